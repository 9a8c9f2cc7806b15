// gdn_scan.cu -- the selective scan's forward (packed, and over pool slots), its state pass over the
// segments of a split scan, and the step of one token for each row.
#include "gdn_scan.cuh"

namespace gdn {
namespace {

// Half of a block's warps ("formers") form d, d x and the outputs, the others ("walkers") walk the
// states, up to 16 of a channel a thread.  While one tile is walked the next one is formed, the
// outputs of the one before are written and the inputs of the one after next are on their way.
template <int NS>
struct WalkShape {
    static constexpr int S = NS < 16 ? NS : 16, L = NS / S;   // states of a walker, walkers of a channel
    static constexpr int kHalf = 128;                         // threads of either kind
    static constexpr int CB = kHalf / L;                      // channels of a block
    static constexpr int TT = 16;                             // tokens of a tile
    static constexpr int kRing = 4;                           // tiles of inputs: finished, walked, formed, on their way
};

template <typename T, int NS, bool kEnds>
struct ScanTiles {
    static constexpr int CB = WalkShape<NS>::CB, TT = WalkShape<NS>::TT, kRing = WalkShape<NS>::kRing;
    float d[2][TT][CB], dx[2][TT][CB];   // d and d x, channels at channel_at
    float B[2][TT][NS], C[2][kEnds ? 1 : TT][NS];
    float y[2][kEnds ? 1 : TT][CB];
    float bias[CB], skip[CB];
    alignas(16) T x[kRing][TT * CB], dt[kRing][TT * CB], z[kEnds ? 1 : kRing][TT * CB];
    alignas(16) T rB[kRing][TT * NS], rC[kEnds ? 1 : kRing][TT * NS];
};

// Runs of four channels change places, so that formers that write eight each meet no bank twice.
__device__ __forceinline__ int channel_at(int c) { return c ^ (c >> 3 & 4); }

// kEnds: the state pass alone (no outputs), for the segments that have another one behind them.
template <typename T, int NS, bool kWide, bool kEnds>
__global__ void __launch_bounds__(2 * WalkShape<NS>::kHalf, 2)
    k_scan_fwd(const __grid_constant__ ScanArgs a) {
    using Shape = WalkShape<NS>;
    constexpr int CB = Shape::CB, L = Shape::L, S = Shape::S, TT = Shape::TT, R = Shape::kRing, EV = 8;
    constexpr int kHalf = Shape::kHalf;
    using Tile = TileOf<T, CB, TT, EV, kHalf, kWide>;
    using Rows = RowsOf<T, NS, TT, kHalf, kWide>;
    using Tiles = ScanTiles<T, NS, kEnds>;
    extern __shared__ float4 smem[];
    Tiles &m = *reinterpret_cast<Tiles *>(smem);

    ScanPlace w;
    if (!scan_place<CB>(a, blockIdx.x, &w)) {
        if (!kEnds && a.pack.status && w.item == a.pack.N + a.pack.T / a.seg) check_offsets(a.pack);
        return;
    }
    if (kEnds && w.seg == w.segs - 1) return;
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
        const bool gated = a.z != nullptr;
        Feed x(static_cast<const T *>(a.x), a.xs, a, w, TT), dt(static_cast<const T *>(a.dt), a.dts, a, w, TT);
        Feed z(static_cast<const T *>(a.z), a.zs, a, w, TT);
        RowFeed B(static_cast<const T *>(a.B), a.bs, a, w, TT), C(static_cast<const T *>(a.Cm), a.cs, a, w, TT);
        const int col = Tile::col();
        auto place = [&](T (*ring)[TT * CB], int i) { return reinterpret_cast<V *>(ring[i % R]); };
        auto fetch = [&](int i) {
            if (i < tiles) {
                x.next(place(m.x, i), a, w, TT);
                dt.next(place(m.dt, i), a, w, TT);
                B.next(reinterpret_cast<U *>(m.rB[i % R]), a, TT);
                if (!kEnds) {
                    if (gated) z.next(place(m.z, i), a, w, TT);
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
                const V xv = place(m.x, i)[Tile::thread() + k * kHalf], dv = place(m.dt, i)[Tile::thread() + k * kHalf];
                const bool there = w.b + i * TT + row < w.f;
                float d4[EV], dx4[EV];
#pragma unroll
                for (int j = 0; j < EV; j += 2) {
                    float2 d = softplus_of(add2(make_float2(as_float(dv.x[j]), as_float(dv.x[j + 1])),
                                                *reinterpret_cast<const float2 *>(&m.bias[col + j])));
                    if (!there) d = both(0.f);
                    const float2 dx = mul2(d, make_float2(as_float(xv.x[j]), as_float(xv.x[j + 1])));
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
            }
            Rows::keep_copied(reinterpret_cast<const U *>(m.rB[i % R]), m.B[i & 1]);
            if (!kEnds) Rows::keep_copied(reinterpret_cast<const U *>(m.rC[i % R]), m.C[i & 1]);
        };
        auto finish = [&](int i) {
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k);
                if (row >= TT) break;
                const V xv = place(m.x, i)[Tile::thread() + k * kHalf];
                V zv, out;
                if (gated) zv = place(m.z, i)[Tile::thread() + k * kHalf];
                const float *sums = m.y[i & 1][row] + col;
#pragma unroll
                for (int j = 0; j < EV; j += 2) {
                    float2 y = fma2(*reinterpret_cast<const float2 *>(&m.skip[col + j]),
                                    make_float2(as_float(xv.x[j]), as_float(xv.x[j + 1])),
                                    *reinterpret_cast<const float2 *>(&sums[j]));
                    if (gated) y = mul2(y, silu_of(make_float2(as_float(zv.x[j]), as_float(zv.x[j + 1]))));
                    out.x[j] = as_type<T>(y.x);
                    out.x[j + 1] = as_type<T>(y.y);
                }
                Tile::store(static_cast<T *>(a.y), a, w, w.b + i * TT, w.f, k, out);
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
            if (!kEnds && i > 0) finish(i - 1);
            __syncthreads();
        }
        return;
    }

    using Lane = ScanLane<NS, 1, S, kHalf>;
    constexpr int H = S / 2;
    const Lane lane(a, w);
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    const int last = w.item - w.seg + w.segs - 1;   // the item of the sequence's last segment
    // The state ahead of the segment.  The record of the last segment, which has no end to keep, holds
    // the state ahead of the sequence: a slot is read once, before any block writes it.
    typename Lane::States h;
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
    float total = 0.f;
    const int place = channel_at(lane.at);
    __syncthreads();
    for (int i = 0; i <= tiles; ++i) {
        if (i < tiles) {
            const float *d = m.d[i & 1][0] + place, *dx = m.dx[i & 1][0] + place;
            const float4 *B = reinterpret_cast<const float4 *>(m.B[i & 1][0] + S * lane.q);
            const float4 *C = reinterpret_cast<const float4 *>(m.C[i & 1][0] + S * lane.q);
            float *y = m.y[i & 1][0] + lane.at;
            float sum = 0.f;
            // All of the tile's tokens: those past the segment change nothing.  The decays, B and C are
            // formed and read one token ahead of the states that take them.
            float2 in = make_float2(d[0], dx[0]), dec[H], b[H], c[H];
            auto ahead = [&](int t) {
#pragma unroll
                for (int k = 0; k < H; k += 2) {
                    const float4 v = B[(t * NS + 2 * k) / 4];
                    b[k] = make_float2(v.x, v.y);
                    b[k + 1] = make_float2(v.z, v.w);
                    if (!kEnds) {
                        const float4 u = C[(t * NS + 2 * k) / 4];
                        c[k] = make_float2(u.x, u.y);
                        c[k + 1] = make_float2(u.z, u.w);
                    }
                }
            };
#pragma unroll
            for (int k = 0; k < H; ++k) dec[k] = lane.decay(0, k, both(in.x));
            ahead(0);
            float2 next = make_float2(d[CB], dx[CB]);
#pragma unroll 8
            for (int t = 0; t < TT; ++t) {
                float2 y2[2] = {both(0.f), both(0.f)};
                const float2 input = both(in.y);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    h[0][k] = fma2(dec[k], h[0][k], mul2(input, b[k]));
                    if (!kEnds) y2[k & 1] = fma2(c[k], h[0][k], y2[k & 1]);
                }
                if (kEnds) sum += in.x;
                const int u = min(t + 1, TT - 1);
                in = next;
                next = make_float2(d[min(t + 2, TT - 1) * CB], dx[min(t + 2, TT - 1) * CB]);
                ahead(u);
#pragma unroll
                for (int k = 0; k < H; ++k) dec[k] = lane.decay(0, k, both(in.x));
                if (!kEnds) {
                    const float2 y1 = add2(y2[0], y2[1]);
                    float out = y1.x + y1.y;
#pragma unroll
                    for (int o = L / 2; o; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
                    if (L == 1 || lane.q == 0) y[t * CB] = out;
                }
            }
            total += sum;
        }
        __syncthreads();
    }
    if (kEnds) {
        lane.store(a.rec_h, w.item, items, a, w, h);
        const long long at = (long long)w.item * a.C + lane.c;
        if (lane.q == 0 && lane.c < w.cend && in_range(at, 1, items * a.C, a.pack.status)) a.rec_d[at] = total;
        return;
    }
    if (w.seg != w.segs - 1) return;
    if (a.slots.idx && a.slots.status && threadIdx.x == kHalf && a.slots.idx[w.n] >= a.slots.num_slots) *a.slots.status = 1;
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

template <typename T, int NS, bool kWide, bool kEnds>
cudaError_t scan_kernel(const ScanArgs &a, cudaStream_t s) {
    const long long blocks = scan_items(a.pack.N, a.pack.T, a.seg) * scan_across<WalkShape<NS>::CB>(a);
    const unsigned grid = (unsigned)(blocks + (!kEnds && a.pack.status ? 1 : 0));
    constexpr int bytes = (int)sizeof(ScanTiles<T, NS, kEnds>), threads = 2 * WalkShape<NS>::kHalf;
    const cudaError_t e = cudaFuncSetAttribute(k_scan_fwd<T, NS, kWide, kEnds>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k_scan_fwd<T, NS, kWide, kEnds><<<grid, threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NS, bool kEnds>
cudaError_t scan(const ScanArgs &a, cudaStream_t s) {
    return scan_wide(a, 8) ? scan_kernel<T, NS, true, kEnds>(a, s) : scan_kernel<T, NS, false, kEnds>(a, s);
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
