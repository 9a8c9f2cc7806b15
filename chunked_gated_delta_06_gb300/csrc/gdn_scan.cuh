// gdn_scan.cuh -- what the selective scan's forward and backward kernels share.
//
// Per channel c (of group g) and state n, with d_t = softplus(dt_t + dt_bias), A = -e^{A_log}:
//   h_t = e^{d_t A} h_{t-1} + d_t x_t B_t[n],   y_t = (sum_n C_t[n] h_t + D x_t) silu(z_t)
//
// A block of 128 threads walks a segment of one sequence for CB channels of one group, a tile of
// tokens at a time.  What is the same for all states of a channel (d, d x, the gate) is formed once,
// element by element over the whole block, and passes through shared memory; in the walk itself a
// thread has two neighbouring channels of four states each, so that a token costs it one 16-byte
// read of (d, d x), one of B and one of C for eight states, and pairs of states are one packed
// product or multiply-add.  The decay is the hardware's 2^x, d (A / ln 2) rounded once.
#pragma once

#include "gdn_mixer.cuh"

namespace gdn {

constexpr int kScanThreads = 128;

template <int NS>
struct ScanShape {
    static constexpr int L = NS / 4;                    // threads of a channel pair
    static constexpr int kPairs = kScanThreads / L;     // channel pairs of a block
    static constexpr int CB = 2 * kPairs;
};

__device__ __forceinline__ unsigned long long as_bits(float2 x) { return *reinterpret_cast<unsigned long long *>(&x); }
__device__ __forceinline__ float2 as_pair(unsigned long long x) { return *reinterpret_cast<float2 *>(&x); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)));
    return as_pair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)));
    return as_pair(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)), "l"(as_bits(c)));
    return as_pair(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 exp2_of(float2 x) { return make_float2(exp2_of(x.x), exp2_of(x.y)); }

// softplus(u) = max(u, 0) + log(1 + e^-|u|), the logarithm as 2 artanh(e / (2 + e)): its series in
// s = e / (2 + e) <= 1/3 up to s^13 is good to 2^-23, for a small e as well (where log(1 + e) from
// a rounded 1 + e would keep nothing of it).
__device__ __forceinline__ float softplus_of(float u) {
    const float e = __expf(-fabsf(u)), s = __fdividef(e, 2.f + e), q = s * s;
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(q, p, 1.f / 9.f);
    p = fmaf(q, p, 1.f / 7.f);
    p = fmaf(q, p, 1.f / 5.f);
    p = fmaf(q, p, 1.f / 3.f);
    p = fmaf(q, p, 1.f);
    return fmaxf(u, 0.f) + 2.f * s * p;
}

// Where a block works.
struct ScanPlace {
    int n, item, seg, segs;      // sequence, its item, the segment and how many the sequence has
    int s, e;                    // the sequence's tokens
    int b, f;                    // the segment's
    int g, c0, cend;             // group, first channel, end of the group's channels
};

__device__ __forceinline__ int first_item(const ScanArgs &a, int n) { return n + offset_of(a.pack, n) / a.seg; }

template <int NS>
__device__ __forceinline__ bool scan_place(const ScanArgs &a, long long block, ScanPlace *p) {
    constexpr int CB = ScanShape<NS>::CB;
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

// A tile's elements of a [T, C] tensor, spread over the block: EV channels of a row in a vector.
template <typename T, int CB, int TT, int EV, bool kWide>
struct TileOf {
    static constexpr int kCols = CB / EV, kVecs = TT * kCols, NV = (kVecs + kScanThreads - 1) / kScanThreads;
    static_assert(kScanThreads % kCols == 0, "a thread's vectors have the same channels");
    using V = Vec<T, EV>;
    static __device__ int row(int k) { return ((int)threadIdx.x + k * kScanThreads) / kCols; }
    static __device__ int col() { return (int)threadIdx.x % kCols * EV; }
    // rows [t, end) of the tile that starts at token t; zeros elsewhere
    static __device__ void load(const T *p, long long stride, const ScanArgs &a, const ScanPlace &w, int t, int end, V (&v)[NV]) {
        const int c = w.c0 + col();
        const long long extent = (a.pack.T - 1) * stride + a.C;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = t + row(k);
            if (kWide) {
                if (row(k) < TT && at < end && c < w.cend) {
                    v[k] = load_vec<EV>(p, at * stride + c, extent, a.pack.status);
                    continue;
                }
#pragma unroll
                for (int i = 0; i < EV; ++i) v[k].x[i] = as_type<T>(0.f);
            } else {
#pragma unroll
                for (int i = 0; i < EV; ++i)
                    v[k].x[i] = row(k) < TT && at < end && c + i < w.cend
                                    ? load_vec<1>(p, at * stride + c + i, extent, a.pack.status).x[0]
                                    : as_type<T>(0.f);
            }
        }
    }
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
template <typename T, int NS, int TT, bool kWide>
struct RowsOf {
    static constexpr int kUnits = TT * NS / 4, NU = (kUnits + kScanThreads - 1) / kScanThreads;
    using V = Vec<T, 4>;
    static __device__ void load(const T *p, long long stride, const ScanArgs &a, const ScanPlace &w, int t, int end, V (&v)[NU]) {
        const long long extent = (a.pack.T - 1) * stride + (long long)a.G * NS;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int u = (int)threadIdx.x + k * kScanThreads, at = t + u / (NS / 4), i = u % (NS / 4) * 4;
            const long long from = at * stride + w.g * NS + i;
            const bool there = u < kUnits && at < end;
            if (kWide && there) {
                v[k] = load_vec<4>(p, from, extent, a.pack.status);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[k].x[j] = there ? load_vec<1>(p, from + j, extent, a.pack.status).x[0] : as_type<T>(0.f);
            }
        }
    }
    static __device__ void keep(const V (&v)[NU], float (*rows)[NS]) {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int u = (int)threadIdx.x + k * kScanThreads;
            if (u >= kUnits) break;
            *reinterpret_cast<float4 *>(&rows[u / (NS / 4)][u % (NS / 4) * 4]) =
                make_float4(as_float(v[k].x[0]), as_float(v[k].x[1]), as_float(v[k].x[2]), as_float(v[k].x[3]));
        }
    }
};

// (d, d x) of two neighbouring channels are one 16-byte unit of a row.  Units are permuted within
// runs of 8, so that threads that write the four units of eight channels meet no bank twice.
__device__ __forceinline__ int unit_at(int unit) { return unit ^ (unit >> 3 & 3); }

// A thread's part of the walk: channels c and c + 1, states 4 q .. 4 q + 3 of each.
template <int NS>
struct ScanLane {
    int pair, q, c;
    float2 A[2][2];      // rates / ln 2, <= 0 and finite (a token without an input has d = 0)
    __device__ ScanLane(const ScanArgs &a, const ScanPlace &w) {
        pair = (int)threadIdx.x / ScanShape<NS>::L;
        q = (int)threadIdx.x % ScanShape<NS>::L;
        c = w.c0 + 2 * pair;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long at = (long long)(c + i) * NS + 4 * q;
            float r[4] = {};
            if (c + i < w.cend && in_range(at, 4, (long long)a.C * NS, a.pack.status))
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = fmaxf(-1.44269504088896341f * expf(a.A_log[at + j]), -3e38f);
            A[i][0] = make_float2(r[0], r[1]);
            A[i][1] = make_float2(r[2], r[3]);
        }
    }
    // the thread's states of a row of [rows, C, NS]
    __device__ void load(const float *p, long long row, long long rows, const ScanArgs &a, const ScanPlace &w, float2 (&h)[2][2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const long long at = (row * a.C + c + i) * NS + 4 * q;
            if (p && row >= 0 && c + i < w.cend && in_range(at, 4, rows * a.C * NS, a.pack.status))
                v = *reinterpret_cast<const float4 *>(p + at);
            h[i][0] = make_float2(v.x, v.y);
            h[i][1] = make_float2(v.z, v.w);
        }
    }
    __device__ void store(float *p, long long row, long long rows, const ScanArgs &a, const ScanPlace &w, const float2 (&h)[2][2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long at = (row * a.C + c + i) * NS + 4 * q;
            if (p && row >= 0 && c + i < w.cend && in_range(at, 4, rows * a.C * NS, a.pack.status))
                *reinterpret_cast<float4 *>(p + at) = make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y);
        }
    }
    __device__ void decays(int i, float d, float2 (&out)[2]) const {
        out[0] = exp2_of(mul2(A[i][0], both(d)));
        out[1] = exp2_of(mul2(A[i][1], both(d)));
    }
    // h <- e^{A sum of d} h + the record of segment `item`
    __device__ void join(const ScanArgs &a, const ScanPlace &w, const float *rec, int item, float2 (&h)[2][2]) const {
        const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
        float2 end[2][2], decay[2];
        load(rec, item, items, a, w, end);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long at = (long long)item * a.C + c + i;
            const float d = c + i < w.cend && in_range(at, 1, items * a.C, a.pack.status) ? a.rec_d[at] : 0.f;
            decays(i, d, decay);
            h[i][0] = fma2(decay[0], h[i][0], end[i][0]);
            h[i][1] = fma2(decay[1], h[i][1], end[i][1]);
        }
    }
};

// Sums over the L threads of a channel pair: K values of each of BT = min(L, 4) tokens come in, and
// thread q has those of token q % BT in v[0].
template <int L, int BT, int K>
__device__ __forceinline__ void pair_sums(float (&v)[BT][K], int q) {
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

template <int NS>
long long scan_across(const ScanArgs &a) {
    return (long long)a.G * ((a.C / a.G + ScanShape<NS>::CB - 1) / ScanShape<NS>::CB);
}

// end states (and sums of d) of every segment but the last of each sequence
cudaError_t launch_scan_ends(const ScanArgs &a, cudaStream_t s);

}  // namespace gdn
