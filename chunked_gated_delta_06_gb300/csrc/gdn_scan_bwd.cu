// gdn_scan_bwd.cu -- gradient of the selective scan (gdn_scan.cuh has the forward's formulas).
//
// With o_t = dy_t silu(z_t), G_t the gradient of h_t and p_t = G_t e^{d_t A} h_{t-1}:
//   G_t = e^{d_{t+1} A} G_{t+1} + C_t o_t
//   dC_t = sum over the group's channels of o_t h_t,      dB_t = the same of G_t d_t x_t
//   dx_t = d_t sum_n G_t B_t + D o_t,                     dd_t = sum_n p_t A + x_t sum_n G_t B_t
//   ddt_t = dd_t softplus'(u_t),                          dA_log = A sum_t p_t d_t
//   dz_t = dy_t (sum_n C_t h_t + D x_t) silu'(z_t)
//
// A walk forward ahead of this one has left the states ahead of each tile in the workspace (the marks).
// A block walks its segment's tiles backwards: the states of a tile are formed again and wait in shared
// memory as e^{dA} h_{t-1}, 32 bytes a thread and token, and each is replaced by the thread's
// dC and dB as the walk back reads it, which the block then adds over its channels.
#include "gdn_scan.cuh"

namespace gdn {
namespace {

constexpr int kScanThreads = 128;

// A thread walks two neighbouring channels of four states each.
template <int NS>
struct PairShape {
    static constexpr int L = NS / 4, kPairs = kScanThreads / L, CB = 2 * kPairs;
    static_assert(CB == 1024 / NS, "as the host counts them");
};
template <int NS, int kFirst = 0>
using PairLane = ScanLane<NS, 2, 4, kFirst>;

// (d, d x) of two neighbouring channels are one 16-byte unit of a row.  Units are permuted within
// runs of 8, so that threads that write the four units of eight channels meet no bank twice.
__device__ __forceinline__ int unit_at(int unit) { return unit ^ (unit >> 3 & 3); }

constexpr int kEV = 4;

template <typename T, int NS>
struct BackTiles {
    static constexpr int CB = PairShape<NS>::CB, TT = kMarkTile, kRing = 4;
    float4 us[2][TT][kScanThreads][2];   // e^{dA} h of a walker's two channels, then its dC and dB
    float4 dd[2][TT][CB / 2];            // d, d x of two channels, at unit_at; then sum G B, sum p A / ln 2
    float4 start[2][kScanThreads];       // of a walker's two channels: the states ahead of the segment
    float os[2][TT][CB];                 // o, then sum C h
    float B[2][TT][NS], C[2][TT][NS];
    float bias[CB], skip[CB];
    alignas(16) T x[kRing][TT * CB], dt[kRing][TT * CB], z[kRing][TT * CB], dy[kRing][TT * CB];
    alignas(16) T rB[kRing][TT * NS], rC[kRing][TT * NS];
};

// As in the forward, half of the threads are formers and half are walkers, a tile apart.
//
// What bounds it: the traffic of shared memory (78 % of the LSU's wavefronts) and the packed fp32.  A state
// takes two exponentials and some 20 products and sums a token here; the sums over states take 18 shuffles of a
// warp for four tokens.  32768 packed tokens of 2048 channels of 16 states, bf16: 1627 us in all, of them this
// kernel 1230, the walk ahead 350, dB and dC's fold 23, the joins 13, the parameters' sums 10; the bytes are 140.
// Walking ahead for the marks, the ends and the starts' gradients in three passes took 1924.  Eight states
// of a channel a thread (half the shuffles) leave one block an SM: slower.
template <typename T, int NS, bool kWide>
__global__ void __launch_bounds__(2 * kScanThreads, 2) k_scan_bwd(const __grid_constant__ ScanArgs a) {
    constexpr int CB = PairShape<NS>::CB, L = PairShape<NS>::L, TT = kMarkTile, BT = L < 4 ? L : 4, N = kScanThreads;
    constexpr int kPairs = PairShape<NS>::kPairs, R = BackTiles<T, NS>::kRing;
    using Tile = TileOf<T, CB, TT, kEV, N, kWide>;
    using Rows = RowsOf<T, NS, TT, N>;
    extern __shared__ float4 smem[];
    BackTiles<T, NS> &m = *reinterpret_cast<BackTiles<T, NS> *>(smem);

    ScanPlace w;
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    if (!scan_place<CB>(a, blockIdx.x, &w)) {
        if (a.pack.status && w.item == items) check_offsets(a.pack);
        // (an idle item's sums)
        const long long from = ((long long)w.item * a.C + w.c0) * (NS + 2), n = min(CB, w.cend - w.c0) * (NS + 2);
        for (int i = threadIdx.x; i < n; i += 2 * N)
            if (w.item < items && in_range(from + i, 1, items * a.C * (NS + 2), a.pack.status)) a.part_c[from + i] = 0.f;
        return;
    }
    for (int i = threadIdx.x; i < CB; i += 2 * N) {
        const bool there = w.c0 + i < w.cend && in_range(w.c0 + i, 1, a.C, a.pack.status);
        m.bias[i] = there && a.dt_bias ? a.dt_bias[w.c0 + i] : 0.f;
        m.skip[i] = there && a.D ? a.D[w.c0 + i] : 0.f;
    }
    __syncthreads();
    const int tiles = (w.f - w.b + TT - 1) / TT;
    const float ln2 = 0.693147180559945309f;
    const long long sums_extent = items * a.C * (NS + 2);

    if (threadIdx.x < N) {
        using V = typename Tile::V;
        using U = typename Rows::V;
        using Feed = FeedOf<Tile, T, N, kWide>;
        using RowFeed = RowFeedOf<Rows, T, NS, N, kWide>;
        const bool gated = a.z != nullptr;
        const int col = Tile::col();
        auto place = [&](T (*ring)[TT * CB], int i) { return reinterpret_cast<V *>(ring[i % R]); };
        auto units = [&](T (*ring)[TT * NS], int i) { return reinterpret_cast<U *>(ring[i % R]); };
        const T *xp = static_cast<const T *>(a.x), *dtp = static_cast<const T *>(a.dt), *Bp = static_cast<const T *>(a.B);
        // d and d x of four channels of a token
        auto form = [&](const V &x, const V &dt, bool there, float4 *dd) {
            float xv[kEV], dv[kEV];
            unpack(x, xv);
            unpack(dt, dv);
#pragma unroll
            for (int j = 0; j < kEV; j += 2) {
                float2 v = softplus_of(add2(make_float2(dv[j], dv[j + 1]), *reinterpret_cast<const float2 *>(&m.bias[col + j])));
                if (!there) v = both(0.f);   // (which leaves the states alone)
                const float2 dx = mul2(v, make_float2(xv[j], xv[j + 1]));
                dd[unit_at((col + j) / 2)] = make_float4(v.x, dx.x, v.y, dx.y);
            }
        };
        // the i-th tile of the walk is the segment's tile tiles - 1 - i
        Feed x(xp, a.xs, a, w, TT), dt(dtp, a.dts, a, w, TT);
        Feed z(static_cast<const T *>(a.z), a.zs, a, w, TT), dy(static_cast<const T *>(a.dy), a.C, a, w, TT);
        RowFeed B(Bp, a.bs, a, w, TT), C(static_cast<const T *>(a.Cm), a.cs, a, w, TT);
        const int skipped = (tiles - 1) * TT;
        x.turn(skipped, TT);
        dt.turn(skipped, TT);
        z.turn(skipped, TT);
        dy.turn(skipped, TT);
        B.turn(skipped, TT);
        C.turn(skipped, TT);
        float dD[kEV] = {}, db[kEV] = {};
        auto fetch = [&](int i) {
            if (i < tiles) {
                x.next(place(m.x, i), a, w, -TT);
                dt.next(place(m.dt, i), a, w, -TT);
                dy.next(place(m.dy, i), a, w, -TT);
                if (gated) z.next(place(m.z, i), a, w, -TT);
                B.next(units(m.rB, i), a, -TT);
                C.next(units(m.rC, i), a, -TT);
            }
            copies_commit();
        };
        auto all = [&](int i) {
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k);
                if (row >= TT) break;
                form(place(m.x, i)[Tile::thread() + k * N], place(m.dt, i)[Tile::thread() + k * N],
                     w.b + (tiles - 1 - i) * TT + row < w.f, m.dd[i & 1][row]);
                float dyv[kEV], zv[kEV];
                unpack(place(m.dy, i)[Tile::thread() + k * N], dyv);
                float2 o[2] = {make_float2(dyv[0], dyv[1]), make_float2(dyv[2], dyv[3])};
                if (gated) {
                    unpack(place(m.z, i)[Tile::thread() + k * N], zv);
#pragma unroll
                    for (int j = 0; j < 2; ++j) o[j] = mul2(o[j], silu_of(make_float2(zv[2 * j], zv[2 * j + 1])));
                }
                *reinterpret_cast<float4 *>(&m.os[i & 1][row][col]) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
            }
            Rows::keep_copied(units(m.rB, i), m.B[i & 1]);
            Rows::keep_copied(units(m.rC, i), m.C[i & 1]);
        };
        const int per_group = a.C / a.G, blocks = (per_group + CB - 1) / CB, mine = (w.c0 - w.g * per_group) / CB;
        auto finish = [&](int i) {
            const int t = w.b + (tiles - 1 - i) * TT;
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k);
                if (row >= TT) break;
                float xv[kEV], dv[kEV], dyv[kEV], zv[kEV], dxv[kEV], ddv[kEV], dzv[kEV];
                unpack(place(m.x, i)[Tile::thread() + k * N], xv);
                unpack(place(m.dt, i)[Tile::thread() + k * N], dv);
                unpack(place(m.dy, i)[Tile::thread() + k * N], dyv);
                if (gated) unpack(place(m.z, i)[Tile::thread() + k * N], zv);
                const bool there = t + row < w.f;
#pragma unroll
                for (int j = 0; j < kEV; j += 2) {
                    const float4 s = m.dd[i & 1][row][unit_at((col + j) / 2)];
                    const float2 gB = make_float2(s.x, s.z), pA = make_float2(s.y, s.w);
                    const float2 xj = make_float2(xv[j], xv[j + 1]);
                    const float2 skip = *reinterpret_cast<const float2 *>(&m.skip[col + j]);
                    float2 o = make_float2(dyv[j], dyv[j + 1]);
                    if (gated) {
                        const float2 zj = make_float2(zv[j], zv[j + 1]);
                        const float2 sig = sigmoid_of(zj), silu = mul2(zj, sig);
                        const float2 slope = fma2(silu, add2(both(1.f), make_float2(-sig.x, -sig.y)), sig);
                        const float2 y = fma2(skip, xj, *reinterpret_cast<const float2 *>(&m.os[i & 1][row][col + j]));
                        const float2 dz = mul2(mul2(o, y), slope);
                        dzv[j] = dz.x;
                        dzv[j + 1] = dz.y;
                        o = mul2(o, silu);
                    }
                    const float2 u = add2(make_float2(dv[j], dv[j + 1]),
                                          *reinterpret_cast<const float2 *>(&m.bias[col + j]));
                    const float2 dxj = fma2(gB, softplus_of(u), mul2(skip, o));
                    const float2 du = mul2(fma2(pA, both(ln2), mul2(gB, xj)), sigmoid_of(u));
                    dxv[j] = dxj.x;
                    dxv[j + 1] = dxj.y;
                    ddv[j] = du.x;
                    ddv[j + 1] = du.y;
                    if (there) {
                        dD[j] = fmaf(o.x, xj.x, dD[j]);
                        dD[j + 1] = fmaf(o.y, xj.y, dD[j + 1]);
                        db[j] += du.x;
                        db[j + 1] += du.y;
                    }
                }
                Tile::store(static_cast<T *>(a.dx), a, w, t, w.f, k, pack<T>(dxv));
                Tile::store(static_cast<T *>(a.ddt), a, w, t, w.f, k, pack<T>(ddv));
                if (gated) Tile::store(static_cast<T *>(a.dz), a, w, t, w.f, k, pack<T>(dzv));
            }
            // dC and dB of the tile over the block's channels: two threads for four states of one of them
            constexpr int kUnits = TT * 2 * L;
            static_assert(kUnits % 16 == 0 && kPairs % 2 == 0, "whole warps take part");
#pragma unroll
            for (int v0 = 0; v0 < kUnits; v0 += N / 2) {
                const int v = v0 + (int)threadIdx.x / 2, part = threadIdx.x % 2;
                if (v >= kUnits) break;
                const int q = v % L, which = v / L % 2, j = v / (2 * L);
                float2 s0 = both(0.f), s1 = s0;
#pragma unroll 8
                for (int p = part; p < kPairs; p += 2) {
                    const int th = p * L + q;
                    const float4 u = m.us[i & 1][j][th][which ^ (th >> 2 & 1)];
                    s0 = add2(s0, make_float2(u.x, u.y));
                    s1 = add2(s1, make_float2(u.z, u.w));
                }
                s0 = add2(s0, make_float2(__shfl_xor_sync(0xffffffffu, s0.x, 1), __shfl_xor_sync(0xffffffffu, s0.y, 1)));
                s1 = add2(s1, make_float2(__shfl_xor_sync(0xffffffffu, s1.x, 1), __shfl_xor_sync(0xffffffffu, s1.y, 1)));
                if (part == 0 && t + j < w.f) {
                    const long long at = (((long long)mine * a.pack.T + t + j) * a.G + w.g) * 2 * NS + which * NS + 4 * q;
                    if (in_range(at, 4, (long long)blocks * a.pack.T * a.G * 2 * NS, a.pack.status))
                        *reinterpret_cast<float4 *>(a.part_bc + at) = make_float4(s0.x, s0.y, s1.x, s1.y);
                }
            }
        };
        fetch(0);
        fetch(1);
        copies_wait<1>();
        if (tiles > 0) all(0);
        __syncthreads();
        for (int i = 0; i <= tiles; ++i) {
            fetch(i + 2);
            copies_wait<1>();
            // (what a thread reads of a finished tile it is the one to write over)
            if (i > 0) finish(i - 1);
            if (i + 1 < tiles) all(i + 1);
            __syncthreads();
        }
        float (*rows)[CB][2] = reinterpret_cast<float (*)[CB][2]>(smem);   // the rows of threads, in order
        constexpr int kRows = N / Tile::kCols;
#pragma unroll
        for (int j = 0; j < kEV; ++j) {
            rows[threadIdx.x / Tile::kCols][col + j][0] = dD[j];
            rows[threadIdx.x / Tile::kCols][col + j][1] = db[j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < CB; i += N) {
            float s[2] = {};
            for (int r = 0; r < kRows; ++r) {
                s[0] += rows[r][i][0];
                s[1] += rows[r][i][1];
            }
            const long long at = ((long long)w.item * a.C + w.c0 + i) * (NS + 2) + NS;
            if (w.c0 + i < w.cend && in_range(at, 2, sums_extent, a.pack.status)) {
                a.part_c[at] = s[0];
                a.part_c[at + 1] = s[1];
            }
        }
        return;
    }

    const PairLane<NS, N> lane(a, w);
    const int me = (int)threadIdx.x - N;
    const long long marks = a.pack.N + (long long)(a.pack.T / kMarkTile), mark = first_mark(a, w);
    // g holds e^{d A} G of the token behind.  h, the states ahead of the tile, is read a tile ahead; in a
    // segment behind another one it is what the segment's start leaves of itself, and the mark.
    const bool behind = w.seg > 0;
    float2 h[2][2], g[2][2], dA[2][2] = {};
    if (w.seg == w.segs - 1) lane.load(a.ds1, w.n, a.pack.N, a, w, g);
    else lane.load(a.rec_g, w.item, items, a, w, g);
    if (behind) {
        lane.load(a.rec_h, w.item, items, a, w, h);
#pragma unroll
        for (int p = 0; p < 2; ++p) m.start[p][me] = make_float4(h[p][0].x, h[p][0].y, h[p][1].x, h[p][1].y);
    }
    float since[2] = {};   // sums of d from the segment's start to the mark
    auto read = [&](int tile, float2 (&to)[2][2]) {
        lane.load(tile >= 0 ? a.marks : nullptr, mark + tile, marks, a, w, to);
        if (!behind || tile < 0) return;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const long long at = (mark + tile) * a.C + lane.c + p;
            since[p] = lane.c + p < w.cend && in_range(at, 1, marks * a.C, a.pack.status) ? a.mark_d[at] : 0.f;
        }
    };
    read(tiles - 1, h);
    __syncthreads();
    for (int i = 0; i <= tiles; ++i) {
        if (i < tiles) {
            if (behind) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float4 s = m.start[p][me];
                    h[p][0] = fma2(lane.decay(p, 0, both(since[p])), make_float2(s.x, s.y), h[p][0]);
                    h[p][1] = fma2(lane.decay(p, 1, both(since[p])), make_float2(s.z, s.w), h[p][1]);
                }
            }
            float2 next[2][2];
            read(tiles - 2 - i, next);
            float4 (*us)[2] = &m.us[i & 1][0][me];   // a token is N of them apart
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const float4 in = m.dd[i & 1][j][unit_at(lane.at)];
                const float4 b = *reinterpret_cast<const float4 *>(&m.B[i & 1][j][4 * lane.q]);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 d = both(p ? in.z : in.x), dx = both(p ? in.w : in.y);
                    const float2 u0 = mul2(lane.decay(p, 0, d), h[p][0]), u1 = mul2(lane.decay(p, 1, d), h[p][1]);
                    us[j * N][p ^ (me >> 2 & 1)] = make_float4(u0.x, u0.y, u1.x, u1.y);
                    h[p][0] = fma2(dx, make_float2(b.x, b.y), u0);
                    h[p][1] = fma2(dx, make_float2(b.z, b.w), u1);
                }
            }
#pragma unroll
            for (int j0 = TT - BT; j0 >= 0; j0 -= BT) {
                float part[BT][6];   // of each token: sum G B, sum p A / ln 2, sum C h of the two channels
#pragma unroll
                for (int jj = BT - 1; jj >= 0; --jj) {
                    const int j = j0 + jj;
                    const float4 in = m.dd[i & 1][j][unit_at(lane.at)];
                    const float2 o = *reinterpret_cast<const float2 *>(&m.os[i & 1][j][2 * lane.at]);
                    const float4 bb = *reinterpret_cast<const float4 *>(&m.B[i & 1][j][4 * lane.q]);
                    const float4 cc = *reinterpret_cast<const float4 *>(&m.C[i & 1][j][4 * lane.q]);
                    const float2 b[2] = {make_float2(bb.x, bb.y), make_float2(bb.z, bb.w)};
                    const float2 c[2] = {make_float2(cc.x, cc.y), make_float2(cc.z, cc.w)};
                    float2 dC[2], dB[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 d = both(p ? in.z : in.x), dx = both(p ? in.w : in.y), op = both(p ? o.y : o.x);
                        const float4 uu = us[j * N][p ^ (me >> 2 & 1)];
                        const float2 u[2] = {make_float2(uu.x, uu.y), make_float2(uu.z, uu.w)};
                        float2 sB, sA, sC;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 hk = fma2(dx, b[k], u[k]);
                            const float2 G = fma2(c[k], op, g[p][k]);
                            const float2 pk = mul2(G, u[k]);
                            dC[k] = p ? fma2(op, hk, dC[k]) : mul2(op, hk);
                            dB[k] = p ? fma2(dx, G, dB[k]) : mul2(dx, G);
                            sB = k ? fma2(G, b[k], sB) : mul2(G, b[k]);
                            sA = k ? fma2(pk, lane.A[p][k], sA) : mul2(pk, lane.A[p][k]);
                            sC = k ? fma2(c[k], hk, sC) : mul2(c[k], hk);
                            dA[p][k] = fma2(pk, d, dA[p][k]);
                            g[p][k] = mul2(lane.decay(p, k, d), G);
                        }
                        part[jj][p] = sB.x + sB.y;
                        part[jj][2 + p] = sA.x + sA.y;
                        part[jj][4 + p] = sC.x + sC.y;
                    }
                    us[j * N][me >> 2 & 1] = make_float4(dC[0].x, dC[0].y, dC[1].x, dC[1].y);
                    us[j * N][1 ^ (me >> 2 & 1)] = make_float4(dB[0].x, dB[0].y, dB[1].x, dB[1].y);
                }
                lane_sums<L, BT, 6>(part, lane.q);
                // (the pair's threads, all of this warp, have read what this takes the place of)
                __syncwarp();
                if (lane.q < BT) {
                    m.dd[i & 1][j0 + lane.q][unit_at(lane.at)] = make_float4(part[0][0], part[0][2], part[0][1], part[0][3]);
                    *reinterpret_cast<float2 *>(&m.os[i & 1][j0 + lane.q][2 * lane.at]) = make_float2(part[0][4], part[0][5]);
                }
            }
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < 2; ++k) h[p][k] = next[p][k];
        }
        __syncthreads();
    }
    __syncthreads();
    if (w.seg == 0 && a.ds0) lane.store(a.ds0, w.n, a.pack.N, a, w, g);
    // the segment's sums for the parameters, [items, C, NS + 2]
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const long long at = ((long long)w.item * a.C + lane.c + p) * (NS + 2) + 4 * lane.q;
        if (lane.c + p >= w.cend || !in_range(at, 4, sums_extent, a.pack.status)) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            a.part_c[at + 2 * k] = dA[p][k].x * lane.A[p][k].x * ln2;
            a.part_c[at + 2 * k + 1] = dA[p][k].y * lane.A[p][k].y * ln2;
        }
    }
}

// dB and dC: the blocks' sums in their order, rounded once.
template <typename T, int NS>
__global__ void __launch_bounds__(256) k_scan_bc(const __grid_constant__ ScanArgs a, int blocks) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4, n = (long long)a.pack.T * a.G * 2 * NS;
    if (i >= n) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) {
        const Vec<float, 4> v = load_vec<4>(a.part_bc, b * n + i, blocks * n, a.pack.status);
        s.x += v.x[0];
        s.y += v.x[1];
        s.z += v.x[2];
        s.w += v.x[3];
    }
    const long long row = i / (2 * NS);
    const int k = (int)(i % (2 * NS));
    T *out = static_cast<T *>(k < NS ? a.dC : a.dB);
    store_vec<4>(out, row * NS + k % NS, (long long)a.pack.T * a.G * NS, a.pack.status,
                 Vec<T, 4>{{as_type<T>(s.x), as_type<T>(s.y), as_type<T>(s.z), as_type<T>(s.w)}});
}

// dA_log, dD and ddt_bias: the items' sums, 32 columns a block, and 32 groups that take every 32nd item in
// order; then the groups in order.
constexpr int kSumGroups = 32;
__global__ void __launch_bounds__(32 * kSumGroups) k_scan_params(const __grid_constant__ ScanArgs a) {
    __shared__ float sums[kSumGroups][33];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5, per = a.Ns + 2;
    const long long i = (long long)blockIdx.x * 32 + lane, n = (long long)a.C * per;
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    float s = 0.f;
#pragma unroll 4
    for (long long k = group; k < items; k += kSumGroups)
        if (i < n && in_range(k * n + i, 1, items * n, a.pack.status)) s += a.part_c[k * n + i];
    sums[group][lane] = s;
    __syncthreads();
    if (group || i >= n) return;
#pragma unroll
    for (int g = 1; g < kSumGroups; ++g) s += sums[g][lane];
    const int c = (int)(i / per), k = (int)(i % per);
    if (k < a.Ns) a.dA_log[(long long)c * a.Ns + k] = s;
    else if (k == a.Ns && a.dD) a.dD[c] = s;
    else if (k == a.Ns + 1 && a.ddt_bias) a.ddt_bias[c] = s;
}

template <typename T, int NS, bool kWide>
cudaError_t bwd(const ScanArgs &a, cudaStream_t s) {
    constexpr int CB = PairShape<NS>::CB;
    constexpr int bytes = (int)sizeof(BackTiles<T, NS>);
    static_assert(kScanThreads / (CB / kEV) * CB * 8 <= sizeof(BackTiles<T, NS>::us), "the last sums fit the states' place");
    const long long blocks = scan_items(a.pack.N, a.pack.T, a.seg) * scan_across<PairShape<NS>::CB>(a);
    cudaError_t e = cudaFuncSetAttribute(k_scan_bwd<T, NS, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k_scan_bwd<T, NS, kWide><<<(unsigned)(blocks + (a.pack.status ? 1 : 0)), 2 * kScanThreads, bytes, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long units = (long long)a.pack.T * a.G * 2 * NS / 4;
    if (units > 0) k_scan_bc<T, NS><<<(unsigned)((units + 255) / 256), 256, 0, s>>>(a, (a.C / a.G + CB - 1) / CB);
    k_scan_params<<<(unsigned)(((long long)a.C * (NS + 2) + 31) / 32), 32 * kSumGroups, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t bwd_of(const ScanArgs &a, cudaStream_t s) {
    return scan_wide(a, kEV) ? bwd<T, NS, true>(a, s) : bwd<T, NS, false>(a, s);
}

}  // namespace

int scan_mark_tile() { return kMarkTile; }

cudaError_t launch_scan_bwd(const ScanArgs &a, cudaStream_t s) {
    cudaError_t e = launch_scan_marks(a, s);
    if (a.seg <= a.pack.T) {
        if (e == cudaSuccess) e = launch_scan_join(a, false, s);
        if (e == cudaSuccess) e = launch_scan_join(a, true, s);
    }
    if (e != cudaSuccess) return e;
    if (a.f32) return a.Ns == 8 ? bwd_of<float, 8>(a, s) : a.Ns == 16 ? bwd_of<float, 16>(a, s) : bwd_of<float, 32>(a, s);
    return a.Ns == 8 ? bwd_of<bf16, 8>(a, s) : a.Ns == 16 ? bwd_of<bf16, 16>(a, s) : bwd_of<bf16, 32>(a, s);
}

}  // namespace gdn
