// gdn_scan.cuh -- what the selective scan's forward and backward kernels share.
//
// Per channel c (of group g) and state n, with d_t = softplus(dt_t + dt_bias), A = -e^{A_log}:
//   h_t = e^{d_t A} h_{t-1} + d_t x_t B_t[n],   y_t = (sum_n C_t[n] h_t + D x_t) silu(z_t)
//
// A block walks a segment of one sequence for CB channels of one group, a tile of tokens at a time.
// What is the same for all states of a channel (d, d x, the gate) is formed once, element by element
// over many threads, and passes through shared memory to the threads that walk the states.  Pairs
// of states are one packed product or multiply-add; the decay is the hardware's 2^x, d (A / ln 2)
// rounded once.
#pragma once

#include "gdn_mixer.cuh"

namespace gdn {

// softplus(u) = max(u, 0) + log(1 + e^-|u|), the logarithm as 2 artanh(s) with s = e / (2 + e) <= 1/3, good
// for a small e as well (where log(1 + e) from a rounded 1 + e would keep nothing of it).  artanh(s) / s is
// a polynomial of s^2 fitted to the function at Chebyshev nodes, reweighted until its relative error is
// level: 1e-8 with five coefficients (the Taylor series takes seven for 1e-8).
__device__ __forceinline__ float softplus_of(float u) {
    const float e = exp_of(-fabsf(u)), s = e * reciprocal_of(2.f + e), q = s * s;
    float p = fmaf(q, 0.14089163f, 0.13980302f);
    p = fmaf(q, p, 0.20012455f);
    p = fmaf(q, p, 0.33333157f);
    p = fmaf(q, p, 1.f);
    return fmaxf(u, 0.f) + 2.f * s * p;
}

// Of two numbers at once, without the larger of the number and 0 (to be added last).
__device__ __forceinline__ float2 softplus_rest(float2 u) {
    const float2 e = exp_of(make_float2(-fabsf(u.x), -fabsf(u.y)));
    const float2 n = add2(e, both(2.f));
    const float2 s = mul2(e, reciprocal_of(n)), q = mul2(s, s);
    float2 p = fma2(q, both(0.14089163f), both(0.13980302f));
    p = fma2(q, p, both(0.20012455f));
    p = fma2(q, p, both(0.33333157f));
    p = fma2(q, p, both(1.f));
    return mul2(add2(s, s), p);
}
__device__ __forceinline__ float2 softplus_of(float2 u) {
    return add2(softplus_rest(u), make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
}
__device__ __forceinline__ float2 silu_of(float2 z) {
    return mul2(z, sigmoid_of(z));
}

// Where a block works.
struct ScanPlace {
    int n, item, seg, segs;      // sequence, its item, the segment and how many the sequence has
    int s, e;                    // the sequence's tokens
    int b, f;                    // the segment's
    int g, c0, cend;             // group, first channel, end of the group's channels
};

__device__ __forceinline__ int first_item(const ScanArgs &a, int n) { return n + offset_of(a.pack, n) / a.seg; }

constexpr int kMarkTile = 8;   // tokens of a tile of the gradient's walk; the states ahead of each are its marks
// (the marks of a sequence follow n + s / tile, as the items of a scan do; a segment is whole tiles)
__device__ __forceinline__ long long first_mark(const ScanArgs &a, const ScanPlace &w) {
    return (long long)w.n + w.s / kMarkTile + (w.b - w.s) / kMarkTile;
}

template <int CB>   // channels of a block
__device__ __forceinline__ bool scan_place(const ScanArgs &a, long long block, ScanPlace *p) {
    const int per_group = a.C / a.G, blocks = (per_group + CB - 1) / CB, across = a.G * blocks;
    const int col = (int)(block % across);
    p->item = (int)(block / across);
    p->g = col / blocks;
    p->c0 = p->g * per_group + col % blocks * CB;
    p->cend = (p->g + 1) * per_group;
    int lo = 0, hi = a.pack.N - 1;
    while (lo < hi) {
        const int mid = (int)(((unsigned)lo + (unsigned)hi + 1) / 2);
        if (first_item(a, mid) <= p->item) lo = mid;
        else hi = mid - 1;
    }
    p->n = lo;
    p->s = offset_of(a.pack, lo);
    p->e = max(p->s, offset_of(a.pack, lo + 1));
    p->segs = max(1, (int)(((long long)p->e - p->s + a.seg - 1) / a.seg));
    p->seg = p->item - first_item(a, lo);
    p->b = (int)min((long long)p->s + (long long)max(p->seg, 0) * a.seg, (long long)p->e);
    p->f = (int)min((long long)p->b + a.seg, (long long)p->e);
    return p->seg >= 0 && p->seg < p->segs;
}

// A tile's elements of a [T, C] tensor, spread over N threads: EV channels of a row in a vector.
template <typename T, int CB, int TT, int EV, int N, bool kWide>
struct TileOf {
    static constexpr int kCols = CB / EV, kVecs = TT * kCols, NV = (kVecs + N - 1) / N;
    static_assert(N % kCols == 0, "a thread's vectors have the same channels");
    using V = Vec<T, EV>;
    static __device__ int thread() { return (int)threadIdx.x % N; }
    static __device__ int row(int k) { return (thread() + k * N) / kCols; }
    static __device__ int col() { return thread() % kCols * EV; }
    // vector k of the tile that starts at token t, where its row is ahead of `end`
    static __device__ void store(T *p, const ScanArgs &a, const ScanPlace &w, int t, int end, int k, const V &v) {
        const int c = w.c0 + col(), at = t + row(k);
        const long long extent = (long long)a.pack.T * a.C;
        if (row(k) >= TT || at >= end) return;
        if (kWide) {
            if (c < w.cend) store_vec<EV>(p, (long long)at * a.C + c, extent, a.pack.status, v);
        } else {
#pragma unroll
            for (int i = 0; i < EV; ++i)
                if (c + i < w.cend) store_vec<1>(p, (long long)at * a.C + c + i, extent, a.pack.status, Vec<T, 1>{{v.x[i]}});
        }
    }
};

// A tile's rows of B or C ([T, G, NS]), four elements a unit.
template <typename T, int NS, int TT, int N>
struct RowsOf {
    static constexpr int kUnits = TT * NS / 4, NU = (kUnits + N - 1) / N;
    using V = Vec<T, 4>;
    static __device__ void keep_copied(const V *v, float (*rows)[NS]) {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int u = (int)threadIdx.x % N + k * N;
            if (u >= kUnits) break;
            float f[4];
            unpack(v[u], f);
            *reinterpret_cast<float4 *>(&rows[u / (NS / 4)][u % (NS / 4) * 4]) = make_float4(f[0], f[1], f[2], f[3]);
        }
    }
};

// Copies tile after tile of a tensor into the thread's own places to[thread + k N] of shared memory.
template <typename Tile, typename T, int N, bool kWide>
struct FeedOf {
    const T *p, *at;
    long long step, apart, extent;
    int left;            // tokens that the segment has from the next tile on
    bool there;
    __device__ FeedOf(const T *from, long long stride, const ScanArgs &a, const ScanPlace &w, int tokens) {
        const int c = w.c0 + Tile::col();
        p = from;
        step = tokens * stride;
        apart = (long long)(N / Tile::kCols) * stride;
        extent = (a.pack.T - 1) * stride + a.C;
        left = w.f - w.b;
        there = from != nullptr && c < w.cend;
        at = from + (long long)(w.b + Tile::row(0)) * stride + c;
    }
    // on to the tile `tokens` on, to walk back from there
    __device__ void turn(int tokens, int tile) {
        at += step / tile * tokens;
        left -= tokens;
        step = -step;
    }
    // tokens: of a tile, negative for a walk back
    __device__ void next(typename Tile::V *to, const ScanArgs &a, const ScanPlace &w, int tokens) {
        // (in a walk forward or back every row of a tile is one of its `tokens`)
        constexpr int E = sizeof(to->x) / sizeof(T), kBytes = (int)sizeof(to->x) > 16 ? 16 : (int)sizeof(to->x);
        constexpr int kE = kBytes / (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < Tile::NV; ++k) {
            if (Tile::thread() + k * N >= Tile::kVecs) break;   // (the tile has fewer vectors than there are threads)
            const T *from = at + k * apart;
            typename Tile::V *place = to + Tile::thread() + k * N;
            const bool row = there && Tile::row(k) < left;
            if (kWide) {
                const bool ok = row && in_range(from - p, E, extent, a.pack.status);
#pragma unroll
                for (int i = 0; i < E; i += kE) copy_async<kBytes>(place->x + i, ok ? from + i : p, ok);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    place->x[i] = row && w.c0 + Tile::col() + i < w.cend && in_range(from - p + i, 1, extent, a.pack.status)
                                      ? from[i]
                                      : as_type<T>(0.f);
            }
        }
        at += step;
        left -= tokens;
    }
};
// The same for the rows of B or C, four elements a unit.
template <typename Rows, typename T, int NS, int N, bool kWide>
struct RowFeedOf {
    const T *p, *at;
    long long step, apart, extent;
    int left;
    __device__ RowFeedOf(const T *from, long long stride, const ScanArgs &a, const ScanPlace &w, int tokens) {
        const int u = (int)threadIdx.x % N;
        p = from;
        step = tokens * stride;
        apart = (long long)(N / (NS / 4)) * stride;
        extent = (a.pack.T - 1) * stride + (long long)a.G * NS;
        left = w.f - w.b;
        at = from + (long long)(w.b + u / (NS / 4)) * stride + w.g * NS + u % (NS / 4) * 4;
    }
    __device__ void turn(int tokens, int tile) {
        at += step / tile * tokens;
        left -= tokens;
        step = -step;
    }
    __device__ void next(typename Rows::V *to, const ScanArgs &a, int tokens) {
        static_assert(N % (NS / 4) == 0, "a thread's units are of the same states");
#pragma unroll
        for (int k = 0; k < Rows::NU; ++k) {
            const int u = (int)threadIdx.x % N + k * N;
            if (u >= Rows::kUnits) break;
            const T *from = at + k * apart;
            const bool ok = u / (NS / 4) < left && in_range(from - p, 4, extent, a.pack.status);
            if (kWide) {
                copy_async<4 * (int)sizeof(T)>(to + u, ok ? from : p, ok);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) to[u].x[i] = ok ? from[i] : as_type<T>(0.f);
            }
        }
        at += step;
        left -= tokens;
    }
};

// The hardware's 2^x is low on average where a state's memory is long (by 5e-9 for x in -0.004 .. 0, up to
// 2.6e-8 below; rms 3e-8), and that adds up over a state's tokens: one of 124 tokens was off by 1.5e-6.
// An argument larger by this leaves 1.1e-8 of either sign at most (and that state 7e-7 off, as one with
// rounded exponentials is); 2 to its own power is still 1, so that a token without a step decays nothing.
constexpr float kLift = 2.2e-8f;

// A / ln 2, kept finite, so that a token without an input (d = 0) decays nothing; NaN stays NaN.
__device__ __forceinline__ float rate_of(float A_log) {
    const float r = -1.44269504088896341f * expf(A_log);
    return r < -3e38f ? -3e38f : r;
}

// A thread's part of a walk: channels c .. c + P - 1, states S q .. S q + S - 1 of each.
template <int NS, int P, int S, int kFirst = 0>   // kFirst: the first thread that walks
struct ScanLane {
    static constexpr int L = NS / S, H = S / 2;
    using States = float2[P][H];
    int at, q, c;        // its group of P channels in the block, its part of the states, its first channel
    float2 A[P][H];      // rate_of its A_log
    __device__ ScanLane(const ScanArgs &a, const ScanPlace &w) {
        at = ((int)threadIdx.x - kFirst) / L;
        q = ((int)threadIdx.x - kFirst) % L;
        c = w.c0 + P * at;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const long long from = (long long)(c + i) * NS + S * q;
            const bool there = c + i < w.cend && in_range(from, S, (long long)a.C * NS, a.pack.status);
            auto rate = [&](int j) { return there ? rate_of(a.A_log[from + j]) : 0.f; };
#pragma unroll
            for (int k = 0; k < H; ++k) A[i][k] = make_float2(rate(2 * k), rate(2 * k + 1));
        }
    }
    // the thread's states of a row of [rows, C, NS]
    __device__ void load(const float *p, long long row, long long rows, const ScanArgs &a, const ScanPlace &w, States &h) const {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int k = 0; k < H; k += 2) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const long long from = (row * a.C + c + i) * NS + S * q + 2 * k;
                if (p && row >= 0 && c + i < w.cend && in_range(from, 4, rows * a.C * NS, a.pack.status))
                    v = *reinterpret_cast<const float4 *>(p + from);
                h[i][k] = make_float2(v.x, v.y);
                h[i][k + 1] = make_float2(v.z, v.w);
            }
    }
    __device__ void store(float *p, long long row, long long rows, const ScanArgs &a, const ScanPlace &w, const States &h) const {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int k = 0; k < H; k += 2) {
                const long long to = (row * a.C + c + i) * NS + S * q + 2 * k;
                if (p && row >= 0 && c + i < w.cend && in_range(to, 4, rows * a.C * NS, a.pack.status))
                    *reinterpret_cast<float4 *>(p + to) = make_float4(h[i][k].x, h[i][k].y, h[i][k + 1].x, h[i][k + 1].y);
            }
    }
    __device__ float2 decay(int i, int k, float2 d) const { return exp2_of(fma2(A[i][k], d, both(kLift))); }
};

// Sums over the L threads that share channels: K values of each of BT <= L tokens come in, and thread
// q has those of token q % BT in v[0].
template <int L, int BT, int K>
__device__ __forceinline__ void lane_sums(float (&v)[BT][K], int q) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) {
        if (o >= BT) {
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int k = 0; k < K; ++k) v[i][k] += __shfl_xor_sync(0xffffffffu, v[i][k], o);
        } else {
            const bool up = q & o;
#pragma unroll
            for (int i = 0; i < o; ++i)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float send = up ? v[i][k] : v[i + o][k], mine = up ? v[i + o][k] : v[i][k];
                    v[i][k] = mine + __shfl_xor_sync(0xffffffffu, send, o);
                }
        }
    }
}

// Where the state of a sequence comes from: its row of s0 (or of the pool), -1 for zeros.
__device__ __forceinline__ int scan_start_row(const ScanArgs &a, int n) {
    if (!a.slots.idx) return a.s0 ? n : -1;
    if (a.slots.resume && a.slots.resume[n] == 0) return -1;
    return slot_of(a.slots, n);
}

// Whether rows of 8 elements can be read and written at once, group by group.
inline bool scan_wide(const ScanArgs &a, int elements) {
    const int bytes = a.f32 ? 4 : 2;
    auto ok = [&](const void *p, long long stride, int n) {
        return !p || (reinterpret_cast<uintptr_t>(p) % (bytes * n > 16 ? 16 : bytes * n) == 0 && stride % n == 0);
    };
    return a.C / a.G % elements == 0 && ok(a.x, a.xs, elements) && ok(a.dt, a.dts, elements) && ok(a.z, a.zs, elements) &&
           ok(a.B, a.bs, 4) && ok(a.Cm, a.cs, 4) && ok(a.y, a.C, elements) && ok(a.dy, a.C, elements) &&
           ok(a.dx, a.C, elements) && ok(a.ddt, a.C, elements) && ok(a.dz, a.C, elements);
}

template <int CB>
long long scan_across(const ScanArgs &a) {
    return (long long)a.G * ((a.C / a.G + CB - 1) / CB);
}

// For a gradient: marks, the states ahead of every tile (in a segment behind another one those that it
// has from nothing, with mark_d, the sums of d since its start), and of split sequences the records:
// end states and sums of d of every segment but the last, start gradients of every one but the first,
cudaError_t launch_scan_marks(const ScanArgs &a, cudaStream_t s);
// and then in the place of rec_h the state ahead of each segment, in the place of rec_g (backward) the
// gradient behind each segment but the last.
cudaError_t launch_scan_join(const ScanArgs &a, bool backward, cudaStream_t s);

}  // namespace gdn
