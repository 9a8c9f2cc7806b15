// gdn_scan.cu -- the selective scan's forward (packed, and over pool slots), its state pass over the
// segments of a split scan, and the step of one token for each row.
#include "gdn_scan.cuh"

namespace gdn {
namespace {

// Tokens of a tile: 16 elements of it a thread.
template <int NS>
constexpr int kTile = 2 * NS;

// kEnds: the state pass alone (no outputs), for the segments that have another one behind them.
template <typename T, int NS, bool kWide, bool kEnds>
__global__ void __launch_bounds__(kScanThreads) k_scan_fwd(const __grid_constant__ ScanArgs a) {
    constexpr int CB = ScanShape<NS>::CB, L = ScanShape<NS>::L, TT = kTile<NS>, BT = L < 4 ? L : 4, EV = 8;
    using Tile = TileOf<T, CB, TT, EV, kWide>;
    using Rows = RowsOf<T, NS, TT, kWide>;
    __shared__ float4 dd[TT][CB / 2];
    __shared__ float Bs[TT][NS], Cs[kEnds ? 1 : TT][NS];
    __shared__ float ys[kEnds ? 1 : TT][CB + 8];
    __shared__ float bias[CB], skip[CB];

    ScanPlace w;
    if (!scan_place<NS>(a, blockIdx.x, &w)) {
        if (!kEnds && a.pack.status && w.item == a.pack.N + a.pack.T / a.seg) check_offsets(a.pack);
        return;
    }
    if (kEnds && w.seg == w.segs - 1) return;
    for (int i = threadIdx.x; i < CB; i += kScanThreads) {
        const bool there = w.c0 + i < w.cend && in_range(w.c0 + i, 1, a.C, a.pack.status);
        bias[i] = there && a.dt_bias ? a.dt_bias[w.c0 + i] : 0.f;
        skip[i] = there && a.D ? a.D[w.c0 + i] : 0.f;
    }
    const ScanLane<NS> lane(a, w);
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    const int last = w.item - w.seg + w.segs - 1;   // the item of the sequence's last segment
    // The state ahead of the segment.  The record of the last segment, which has no end to keep, holds
    // the state ahead of the sequence: a slot is read once, before any block writes it.
    float2 h[2][2];
    if (w.seg == 0 && (kEnds || w.segs == 1)) {
        lane.load(a.s0, scan_start_row(a, w.n), a.slots.idx ? a.slots.num_slots : a.pack.N, a, w, h);
        if (kEnds) lane.store(a.rec_h, last, items, a, w, h);
    } else if (kEnds) {
        lane.load(nullptr, -1, 0, a, w, h);
    } else if (w.seg == 0) {
        lane.load(a.rec_h, last, items, a, w, h);
    } else {
        lane.load(a.rec_h, w.item - w.seg, items, a, w, h);
        for (int i = w.item - w.seg + 1; i < w.item; ++i) lane.join(a, w, a.rec_h, i, h);
    }

    const T *x = static_cast<const T *>(a.x), *dt = static_cast<const T *>(a.dt), *z = static_cast<const T *>(a.z);
    const T *B = static_cast<const T *>(a.B), *Cm = static_cast<const T *>(a.Cm);
    typename Tile::V xn[Tile::NV], dn[Tile::NV], zn[Tile::NV];
    typename Rows::V bn[Rows::NU], cn[Rows::NU];
    auto fetch = [&](int t) {
        Tile::load(x, a.xs, a, w, t, w.f, xn);
        Tile::load(dt, a.dts, a, w, t, w.f, dn);
        Rows::load(B, a.bs, a, w, t, w.f, bn);
        if (!kEnds) {
            if (z) Tile::load(z, a.zs, a, w, t, w.f, zn);
            Rows::load(Cm, a.cs, a, w, t, w.f, cn);
        }
    };
    float total[2] = {};
    if (w.b < w.f) fetch(w.b);
    __syncthreads();
    for (int t = w.b; t < w.f; t += TT) {
        // d and d x of the tile; a token past the segment has d = 0, which leaves the state alone
        typename Tile::V xc[Tile::NV], zc[Tile::NV];
#pragma unroll
        for (int k = 0; k < Tile::NV; ++k) {
            const int row = Tile::row(k), col = Tile::col();
            float d[EV];
#pragma unroll
            for (int i = 0; i < EV; ++i)
                d[i] = t + row < w.f && w.c0 + col + i < w.cend ? softplus_of(as_float(dn[k].x[i]) + bias[col + i]) : 0.f;
#pragma unroll
            for (int i = 0; i < EV; i += 2)
                dd[row][unit_at((col + i) / 2)] =
                    make_float4(d[i], d[i] * as_float(xn[k].x[i]), d[i + 1], d[i + 1] * as_float(xn[k].x[i + 1]));
            xc[k] = xn[k];
            if (!kEnds) zc[k] = zn[k];
        }
        Rows::keep(bn, Bs);
        if (!kEnds) Rows::keep(cn, Cs);
        __syncthreads();
        if (t + TT < w.f) fetch(t + TT);
        float sum[2] = {};
        const int tokens = min(TT, w.f - t);
        for (int i0 = 0; i0 < tokens; i0 += BT) {
            float part[BT][2];
#pragma unroll
            for (int i = 0; i < BT; ++i) {
                const float4 in = dd[i0 + i][unit_at(lane.pair)];
                const float4 b = *reinterpret_cast<const float4 *>(&Bs[i0 + i][4 * lane.q]);
                const float2 b0 = make_float2(b.x, b.y), b1 = make_float2(b.z, b.w);
                float2 c0, c1;
                if (!kEnds) {
                    const float4 c = *reinterpret_cast<const float4 *>(&Cs[i0 + i][4 * lane.q]);
                    c0 = make_float2(c.x, c.y);
                    c1 = make_float2(c.z, c.w);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float d = p ? in.z : in.x, dx = p ? in.w : in.y;
                    float2 decay[2];
                    lane.decays(p, d, decay);
                    h[p][0] = fma2(decay[0], h[p][0], mul2(both(dx), b0));
                    h[p][1] = fma2(decay[1], h[p][1], mul2(both(dx), b1));
                    if (kEnds) {
                        sum[p] += d;
                    } else {
                        const float2 y = fma2(c1, h[p][1], mul2(c0, h[p][0]));
                        part[i][p] = y.x + y.y;
                    }
                }
            }
            if (!kEnds) {
                pair_sums<L, BT, 2>(part, lane.q);
                if (lane.q < BT)
                    *reinterpret_cast<float2 *>(&ys[i0 + lane.q][2 * lane.pair]) = make_float2(part[0][0], part[0][1]);
            }
        }
        if (kEnds) {
            total[0] += sum[0];
            total[1] += sum[1];
        }
        __syncthreads();
        if (!kEnds) {
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k), col = Tile::col();
                typename Tile::V out;
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    float y = fmaf(skip[col + i], as_float(xc[k].x[i]), ys[row][col + i]);
                    if (z) {
                        const float g = as_float(zc[k].x[i]);
                        y *= g * sigmoid_of(g);
                    }
                    out.x[i] = as_type<T>(y);
                }
                Tile::store(static_cast<T *>(a.y), a, w, t, w.f, k, out);
            }
        }
    }
    if (kEnds) {
        lane.store(a.rec_h, w.item, items, a, w, h);
        if (lane.q == 0)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const long long at = (long long)w.item * a.C + lane.c + p;
                if (lane.c + p < w.cend && in_range(at, 1, items * a.C, a.pack.status)) a.rec_d[at] = total[p];
            }
        return;
    }
    if (w.seg != w.segs - 1) return;
    if (a.slots.idx && a.slots.status && threadIdx.x == 0 && a.slots.idx[w.n] >= a.slots.num_slots) *a.slots.status = 1;
    const int to = a.slots.idx ? slot_of(a.slots, w.n) : w.n;
    lane.store(a.s1, to, a.slots.idx ? a.slots.num_slots : a.pack.N, a, w, h);
}

// One token for each row: a thread has four states of one channel.  Bound by HBM, the states read and
// written once.
template <typename T, int NS>
__global__ void __launch_bounds__(256) k_scan_step(const __grid_constant__ ScanArgs a, int across) {
    constexpr int L = NS / 4, CB = 256 / L;
    const int b = blockIdx.x / across, c = (int)(blockIdx.x % across) * CB + (int)threadIdx.x / L, q = threadIdx.x % L;
    const bool there = c < a.C;
    const int slot = slot_of(a.slots, b);
    T *y = static_cast<T *>(a.y);
    const long long extent = (long long)a.pack.T * a.C, to = (long long)b * a.C + c;
    if (slot < 0) {
        if (threadIdx.x == 0 && a.slots.status && a.slots.idx[b] >= a.slots.num_slots) *a.slots.status = 1;
        if (there && q == 0) store_vec<1>(y, to, extent, a.pack.status, Vec<T, 1>{{as_type<T>(0.f)}});
        return;
    }
    float sum = 0.f, x = 0.f;
    if (there) {
        const long long at = ((long long)slot * a.C + c) * NS + 4 * q, n = (long long)a.slots.num_slots * a.C * NS;
        const Vec<float, 4> h = load_vec<4>(a.s1, at, n, a.pack.status);
        const int g = c / (a.C / a.G);
        auto in = [&](const void *p, long long stride) {
            return as_float(load_vec<1>(static_cast<const T *>(p), b * stride + c, (a.pack.T - 1) * stride + a.C, a.pack.status).x[0]);
        };
        x = in(a.x, a.xs);
        const float d = softplus_of(in(a.dt, a.dts) + (a.dt_bias ? a.dt_bias[c] : 0.f));
        Vec<float, 4> out;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = g * NS + 4 * q + j;
            const float bv = as_float(load_vec<1>(static_cast<const T *>(a.B), b * a.bs + s, (a.pack.T - 1) * a.bs + a.G * NS, a.pack.status).x[0]);
            const float cv = as_float(load_vec<1>(static_cast<const T *>(a.Cm), b * a.cs + s, (a.pack.T - 1) * a.cs + a.G * NS, a.pack.status).x[0]);
            const float rate = fmaxf(-1.44269504088896341f * expf(load_vec<1>(a.A_log, (long long)c * NS + 4 * q + j, (long long)a.C * NS, a.pack.status).x[0]), -3e38f);
            out.x[j] = fmaf(exp2_of(d * rate), h.x[j], d * x * bv);
            sum = fmaf(cv, out.x[j], sum);
        }
        store_vec<4>(a.s1, at, n, a.pack.status, out);
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!there || q) return;
    if (a.D) sum = fmaf(a.D[c], x, sum);
    if (a.z) {
        const float z = as_float(load_vec<1>(static_cast<const T *>(a.z), b * a.zs + c, (a.pack.T - 1) * a.zs + a.C, a.pack.status).x[0]);
        sum *= z * sigmoid_of(z);
    }
    store_vec<1>(y, to, extent, a.pack.status, Vec<T, 1>{{as_type<T>(sum)}});
}

template <typename T, int NS, bool kEnds>
cudaError_t scan(const ScanArgs &a, cudaStream_t s) {
    const long long blocks = scan_items(a.pack.N, a.pack.T, a.seg) * scan_across<NS>(a);
    const unsigned grid = (unsigned)(blocks + (!kEnds && a.pack.status ? 1 : 0));
    if (scan_wide(a, 8)) k_scan_fwd<T, NS, true, kEnds><<<grid, kScanThreads, 0, s>>>(a);
    else k_scan_fwd<T, NS, false, kEnds><<<grid, kScanThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t step(const ScanArgs &a, int batch, cudaStream_t s) {
    constexpr int CB = 256 / (NS / 4);
    const int across = (a.C + CB - 1) / CB;
    k_scan_step<T, NS><<<(unsigned)((long long)batch * across), 256, 0, s>>>(a, across);
    return cudaGetLastError();
}

template <bool kEnds>
cudaError_t scan_of(const ScanArgs &a, cudaStream_t s) {
    if (a.f32) return a.Ns == 8 ? scan<float, 8, kEnds>(a, s) : a.Ns == 16 ? scan<float, 16, kEnds>(a, s) : scan<float, 32, kEnds>(a, s);
    return a.Ns == 8 ? scan<bf16, 8, kEnds>(a, s) : a.Ns == 16 ? scan<bf16, 16, kEnds>(a, s) : scan<bf16, 32, kEnds>(a, s);
}

}  // namespace

cudaError_t launch_scan_ends(const ScanArgs &a, cudaStream_t s) { return scan_of<true>(a, s); }

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
    if (a.seg <= a.pack.T) {
        const cudaError_t e = launch_scan_ends(a, s);
        if (e != cudaSuccess) return e;
    }
    return scan_of<false>(a, s);
}

cudaError_t launch_scan_step(const ScanArgs &a, int batch, cudaStream_t s) {
    if (a.f32) return a.Ns == 8 ? step<float, 8>(a, batch, s) : a.Ns == 16 ? step<float, 16>(a, batch, s) : step<float, 32>(a, batch, s);
    return a.Ns == 8 ? step<bf16, 8>(a, batch, s) : a.Ns == 16 ? step<bf16, 16>(a, batch, s) : step<bf16, 32>(a, batch, s);
}

}  // namespace gdn
