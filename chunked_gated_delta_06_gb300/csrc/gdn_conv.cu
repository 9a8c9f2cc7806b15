// gdn_conv.cu -- the short causal convolution of packed sequences: forward (also over pool slots),
// backward and a step of one token for each row.
//
// Channel c of token t, with W weights and what came before the sequence in its state:
//   u_t = bias + sum_j w_j x_{t-(W-1)+j},   y_t = u_t or u_t sigmoid(u_t)
// and with d_t = dy_t y'(u_t):
//   dx_t = sum_j w_j d_{t+(W-1)-j},   dw_j = sum_t d_t x_{t-(W-1)+j},   dbias = sum_t d_t
// The state is the last W - 1 inputs, oldest first, so it has no arithmetic of its own.
#include "gdn_mixer.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

// Where the state of a sequence is read: its row of s0 (or of the pool), -1 for zeros.
__device__ __forceinline__ int start_row(const ConvArgs &a, int n) {
    if (!a.slots.idx) return a.s0 ? n : -1;
    if (a.slots.resume && a.slots.resume[n] == 0) return -1;
    return slot_of(a.slots, n);
}

// Everything of a call that a thread's V channels need again and again.
template <typename T, int V, int W>
struct Channels {
    const ConvArgs &a;
    int c;
    float w[W][V], b[V];
    __device__ Channels(const ConvArgs &args, int channel) : a(args), c(channel) {
        if constexpr (V % 4 == 0) {   // the V channels' weights lie together
            if (reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && in_range((long long)c * W, V * W, (long long)a.C * W, a.pack.status)) {
                float all[V * W];
#pragma unroll
                for (int i = 0; i < V * W / 4; ++i)
                    reinterpret_cast<float4 *>(all)[i] = reinterpret_cast<const float4 *>(a.w + (long long)c * W)[i];
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < W; ++j) w[j][v] = all[v * W + j];
                    b[v] = a.bias ? a.bias[c + v] : 0.f;
                }
                return;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool there = in_range((long long)(c + v) * W, W, (long long)a.C * W, a.pack.status);
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = there ? a.w[(long long)(c + v) * W + j] : 0.f;
            b[v] = a.bias && there ? a.bias[c + v] : 0.f;
        }
    }
    __device__ Vec<T, V> token(const void *x, long long t, long long stride) const {
        return load_vec<V>(static_cast<const T *>(x), t * stride + c, (a.pack.T - 1) * stride + a.C, a.pack.status);
    }
    // V channels' entry k of a state row
    __device__ void state(const void *s, int row, int rows, int k, float (&out)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const long long i = ((long long)row * a.C + c + v) * (W - 1) + k;
            out[v] = row >= 0 && s && in_range(i, 1, (long long)rows * a.C * (W - 1), a.pack.status)
                         ? as_float(static_cast<const T *>(s)[i])
                         : 0.f;
        }
    }
    __device__ int rows() const { return a.slots.idx ? a.slots.num_slots : a.pack.N; }
    // win[k] = x_{t-(W-1)+k} for the sequence n that starts at token s
    __device__ void window(int n, int s, int t, float (&win)[W][V]) const {
        const int row = t - (W - 1) < s ? start_row(a, n) : -1;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int p = t - (W - 1) + k;
            if (p >= s) {
                unpack(token(a.x, p, a.x_stride), win[k]);
            } else {
                state(a.s0, row, rows(), p - s + W - 1, win[k]);
            }
        }
    }
    __device__ void pre(const float (&win)[W][V], float (&u)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = b[v];
#pragma unroll
        for (int j = 0; j < W; ++j) fma_all(u, w[j], win[j]);
    }
    __device__ static void shift(float (&win)[W][V]) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
    }
};

// Channels of a thread that writes states.
template <int V>
constexpr int state_channels() { return V > 1 ? 4 : 1; }
template <int V>
__host__ __device__ int state_blocks(int C) {   // of a sequence
    constexpr int per = kThreads * state_channels<V>();
    return (C + per - 1) / per;
}

// The state behind sequence n for V channels: its last W - 1 inputs, the older ones from the state ahead of it.
// The thread that reads a channel's old state writes the new one, so a slot may hold both.
template <typename T, int V, int W>
__device__ void final_state(const ConvArgs &a, int n, int c) {
    if (c >= a.C || !a.s1) return;
    const int s = offset_of(a.pack, n), e = max(s, offset_of(a.pack, n + 1));
    const int row = start_row(a, n), to = a.slots.idx ? slot_of(a.slots, n) : n;
    const Channels<T, V, W> ch(a, c);
    if (a.slots.idx && c == 0 && a.slots.status && a.slots.idx[n] >= a.slots.num_slots) *a.slots.status = 1;
    if (to < 0) return;
    float flat[W - 1][V];   // the V channels' entries as they lie together
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int p = e - (W - 1) + k;
        float x[V];
        if (p >= s) unpack(ch.token(a.x, p, a.x_stride), x);
        else ch.state(a.s0, row, ch.rows(), p - s + W - 1, x);
#pragma unroll
        for (int v = 0; v < V; ++v) flat[(v * (W - 1) + k) / V][(v * (W - 1) + k) % V] = x[v];
    }
    const long long i = ((long long)to * a.C + c) * (W - 1), extent = (long long)ch.rows() * a.C * (W - 1);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<V>(static_cast<T *>(a.s1), i + k * V, extent, a.pack.status, pack<T>(flat[k]));
}

// A thread's own inputs on their way: `kTensors` rows of V channels a token, kGroup tokens at a time,
// kAhead groups ahead, copied into shared memory asynchronously (so that no registers wait for them).
template <typename T, int V, int kTensors>
struct Stream {
    static constexpr int kGroup = 4, kAhead = 3, kStages = kAhead + 1, kStage = kGroup * kTensors * kThreads;
    using Row = Vec<T, V>;
    Row *ring;                  // the thread's place of [kStages][kGroup][kTensors][threads]
    const T *at[kTensors];      // the next group's first rows
    long long apart[kTensors];
    int left, stage;            // tokens to fetch, where the next group goes
    __device__ const Row &row(int stage, int u, int k) const { return ring[stage * kStage + (u * kTensors + k) * kThreads]; }
    template <typename F>   // in(k, p): whether a row lies in tensor k
    __device__ void fetch(F in) {
        Row *to = ring + stage * kStage;
        auto copy = [&](int u, int k) {
            const T *from = at[k] + u * apart[k];
            if (!in(k, from)) return;
            if constexpr (sizeof(Row) >= 4) copy_async<(int)sizeof(Row)>(to + (u * kTensors + k) * kThreads, from, true);
            else to[(u * kTensors + k) * kThreads] = *reinterpret_cast<const Row *>(from);
        };
        if (left >= kGroup) {
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
#pragma unroll
                for (int k = 0; k < kTensors; ++k) copy(u, k);
        } else {
#pragma unroll 1
            for (int u = 0; u < left; ++u)
#pragma unroll
                for (int k = 0; k < kTensors; ++k) copy(u, k);
        }
        copies_commit();
#pragma unroll
        for (int k = 0; k < kTensors; ++k) at[k] += kGroup * apart[k];
        left -= kGroup;
        stage = stage + 1 < kStages ? stage + 1 : 0;
    }
};

// A thread's channels and tile: a block's are of one tile, or (kFlat, few channels) threads go through a
// tile's channels, then the next tile's.
struct Place {
    int c, tile;
};
template <int V, bool kFlat>
__device__ __forceinline__ Place place_of(const ConvArgs &a, long long block) {
    if (kFlat) {
        const long long i = block * kThreads + threadIdx.x;
        const int per = (a.C + V - 1) / V;
        return {(int)(i % per) * V, (int)(i / per)};
    }
    const int across = (a.C + kThreads * V - 1) / (kThreads * V);
    return {((int)(block % across) * kThreads + (int)threadIdx.x) * V, (int)(block / across)};
}

// A thread walks the tokens of a tile for V channels (16 bytes of them) with the last W - 1 inputs in
// registers, so that an input is read once but for W - 1 of a tile's 64.  Bound by HBM: 32768 packed tokens of
// 8192 channels in bf16, 4 weights, silu, take 170 us, 6.3 TB/s or 0.93 of the copy rate.  (With its loads in
// registers 260 us: a thread had four rows on their way; pairs of channels in one instruction and pointers that
// move with the tokens took it from 174.)  The blocks behind those of the tiles write the states behind the sequences (over a pool they
// are a launch of their own: the tiles still read the slots).
template <typename T, int V, int W, bool kFlat>
__global__ void __launch_bounds__(kThreads) k_conv_fwd(const __grid_constant__ ConvArgs a, long long blocks) {
    using In = Stream<T, V, 1>;
    __shared__ __align__(16) T ring[In::kStages * In::kGroup * kThreads * V];
    const long long block = blockIdx.x;
    if (block >= blocks) {
        constexpr int SV = state_channels<V>();
        const int per = state_blocks<V>(a.C);
        const long long i = block - blocks;
        if (i >= (long long)a.pack.N * per) check_offsets(a.pack);
        else final_state<T, SV, W>(a, (int)(i / per), ((int)(i % per) * kThreads + (int)threadIdx.x) * SV);
        return;
    }
    const Place at = place_of<V, kFlat>(a, block);
    const int c = at.c;
    if (c >= a.C || (long long)at.tile * a.tile >= a.pack.T) return;
    const int t0 = at.tile * a.tile, t1 = (int)min((long long)t0 + a.tile, (long long)a.pack.T);
    const long long extent = (long long)a.pack.T * a.C, x_extent = (a.pack.T - 1) * a.x_stride + a.C;
    const T *x0 = static_cast<const T *>(a.x);
    In in{reinterpret_cast<Vec<T, V> *>(ring) + threadIdx.x, {x0 + t0 * a.x_stride + c}, {a.x_stride}, t1 - t0, 0};
    auto address = [&](int, const T *p) { return in_range(p - x0, V, x_extent, a.pack.status); };
#pragma unroll
    for (int g = 0; g < In::kAhead; ++g) in.fetch(address);
    const Channels<T, V, W> ch(a, c);
    T *y = static_cast<T *>(a.y) + (long long)t0 * a.C + c;
    float win[W][V];
    int end = t0, stage = 0;
    for (int t = t0; t < t1; t += In::kGroup) {
        in.fetch(address);
        copies_wait<In::kAhead>();
        auto one = [&](int u) {
            unpack(in.row(stage, u, 0), win[W - 1]);
            float out[V];
            ch.pre(win, out);
            if (a.silu) {
                float sig[V];
                sigmoid_all(sig, out);
                mul_all(out, out, sig);
            }
            ch.shift(win);
            store_vec<V>(y, 0, extent - (y - static_cast<T *>(a.y)), a.pack.status, pack<T>(out));
            y += a.C;
        };
        if (t != end && t + In::kGroup <= end) {   // (all of one sequence: the window moves by names alone)
#pragma unroll
            for (int u = 0; u < In::kGroup; ++u) one(u);
        } else {
#pragma unroll 1
            for (int u = 0; u < In::kGroup && t + u < t1; ++u) {
                if (t + u == end) {   // the tile's first token, or a sequence's
                    const int n = sequence_of(a.pack, end), s = min(offset_of(a.pack, n), end), e = offset_of(a.pack, n + 1);
                    ch.window(n, s, end, win);
                    end = e > end ? min(e, t1) : t1;
                }
                one(u);
            }
        }
        stage = stage + 1 < In::kStages ? stage + 1 : 0;
    }
}

// A thread walks a tile and the W - 1 tokens behind it: at token t it has d_t and, with the d's
// before, dx of token t - (W - 1) (where that lies ahead of the sequence, of its state's entry); behind
// the last token of a sequence come W - 1 more with d = 0.  Sums for dw and dbias are of the tile's own
// tokens; k_fold adds the tiles.  16384 tokens of 8192 channels, bf16, take 166 us, 4.9 TB/s or 0.72 of the
// copy rate: instructions (issue 60 %) and the registers, which leave four blocks an SM, bound it together.  Tiles of 128 tokens read an eighth less twice than 64; 16 bytes a thread spilled.
template <typename T, int V, int W, bool kFlat>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(const __grid_constant__ ConvArgs a, long long blocks) {
    using In = Stream<T, V, 2>;
    extern __shared__ __align__(16) unsigned char ring[];
    const long long block = blockIdx.x;
    if (block >= blocks) {   // sequences without tokens: the state passed through
        constexpr int SV = state_channels<V>();
        const int per = state_blocks<V>(a.C);
        const long long i = block - blocks;
        if (i >= (long long)a.pack.N * per) {
            check_offsets(a.pack);
            return;
        }
        const int n = (int)(i / per), c = ((int)(i % per) * kThreads + (int)threadIdx.x) * SV;
        if (c >= a.C || !a.ds0 || offset_of(a.pack, n + 1) > offset_of(a.pack, n)) return;
        const long long at = ((long long)n * a.C + c) * (W - 1), extent = (long long)a.pack.N * a.C * (W - 1);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Vec<T, SV> v;
#pragma unroll
            for (int j = 0; j < SV; ++j) v.x[j] = as_type<T>(0.f);
            if (a.ds1) v = load_vec<SV>(static_cast<const T *>(a.ds1), at + k * SV, extent, a.pack.status);
            store_vec<SV>(static_cast<T *>(a.ds0), at + k * SV, extent, a.pack.status, v);
        }
        return;
    }
    const Place place = place_of<V, kFlat>(a, block);
    const int c = place.c, tile = place.tile;
    if (c >= a.C || (long long)tile * a.tile >= a.pack.T) return;
    const int t0 = tile * a.tile, t1 = (int)min((long long)t0 + a.tile, (long long)a.pack.T);
    const int reach = (int)min((long long)t1 + W - 1, (long long)a.pack.T);
    const long long extent = (long long)a.pack.T * a.C, x_extent = (a.pack.T - 1) * a.x_stride + a.C;
    const T *x0 = static_cast<const T *>(a.x), *dy0 = static_cast<const T *>(a.dy);
    In in{reinterpret_cast<Vec<T, V> *>(ring) + threadIdx.x, {x0 + t0 * a.x_stride + c, dy0 + (long long)t0 * a.C + c},
          {a.x_stride, a.C}, reach - t0, 0};
    auto address = [&](int k, const T *p) { return in_range(p - (k ? dy0 : x0), V, k ? extent : x_extent, a.pack.status); };
#pragma unroll
    for (int g = 0; g < In::kAhead; ++g) in.fetch(address);
    const Channels<T, V, W> ch(a, c);
    T *dx = static_cast<T *>(a.dx);
    float dw[W][V] = {}, db[V] = {}, win[W][V] = {}, d[W][V] = {};   // d[k] = d_{t-(W-1)+k}
    int n = 0, s = t0, e = t0, p = t0;   // the sequence and its part of the tile, [p, min(e, t1))
    // dx of token `at`, from the d's of `at` and the W - 1 behind it; past: of a sequence's last ones
    auto emit = [&](int at, bool past) {
        if (at >= min(e, t1) || (at < p && p != s)) return;
        float g[V] = {};   // the final state's gradient: entry k holds input e - (W - 1) + k
        if (past && a.ds1) ch.state(a.ds1, n, a.pack.N, at - e + W - 1, g);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) g[v] = fmaf(ch.w[j][v], d[W - 1 - j][v], g[v]);
        const Vec<T, V> out = pack<T>(g);
        if (at >= p) {
            store_vec<V>(dx, (long long)at * a.C + c, extent, a.pack.status, out);
        } else if (a.ds0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const long long i = ((long long)n * a.C + c + v) * (W - 1) + (at - s + W - 1);
                if (in_range(i, 1, (long long)a.pack.N * a.C * (W - 1), a.pack.status))
                    static_cast<T *>(a.ds0)[i] = out.x[v];
            }
        }
    };
    auto run_out = [&] {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) d[W - 1][v] = 0.f;
            emit(e + i - (W - 1), true);
            ch.shift(d);
        }
    };
    int stage = 0;
    bool open = false;   // a sequence is being walked
    for (int t = t0; t < reach; t += In::kGroup) {
        in.fetch(address);
        copies_wait<In::kAhead>();
        auto one = [&](int u, bool own) {   // d_t, and the sums of the tile's own tokens
            unpack(in.row(stage, u, 0), win[W - 1]);
            unpack(in.row(stage, u, 1), d[W - 1]);
            if (a.silu) {
                float o[V], sig[V], rest[V], one_[V];
                ch.pre(win, o);
                sigmoid_all(sig, o);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    one_[v] = 1.f;
                    rest[v] = -sig[v];
                }
                add_all(rest, one_);
                mul_all(o, o, sig);
                fma_all(sig, o, rest);   // the slope
                mul_all(d[W - 1], d[W - 1], sig);
            }
            if (own) {
#pragma unroll
                for (int j = 0; j < W; ++j) fma_all(dw[j], d[W - 1], win[j]);
                add_all(db, d[W - 1]);
            }
        };
        if (open && t - (W - 1) >= p && t + In::kGroup <= min(e, t1)) {
            // (all of one sequence, every token's dx of the tile: windows move by names alone)
            T *out = dx + (long long)(t - (W - 1)) * a.C + c;
#pragma unroll
            for (int u = 0; u < In::kGroup; ++u) {
                one(u, true);
                float g[V];
                mul_all(g, ch.w[0], d[W - 1]);
#pragma unroll
                for (int j = 1; j < W; ++j) fma_all(g, ch.w[j], d[W - 1 - j]);
                store_vec<V>(out, 0, extent - (out - dx), a.pack.status, pack<T>(g));
                out += a.C;
                ch.shift(win);
                ch.shift(d);
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < In::kGroup && t + u < reach; ++u) {
                const int at = t + u;
                if (at == e) {
                    if (open) run_out();
                    open = at < t1;
                    if (open) {
                        n = sequence_of(a.pack, at);
                        s = min(offset_of(a.pack, n), at);
                        e = offset_of(a.pack, n + 1);
                        e = e > at ? e : t1;
                        p = at;
                        ch.window(n, s, p, win);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k)
#pragma unroll
                            for (int v = 0; v < V; ++v) d[k][v] = 0.f;
                    }
                }
                if (!open) break;
                one(u, at < t1);
                emit(at - (W - 1), false);
                ch.shift(win);
                ch.shift(d);
            }
        }
        stage = stage + 1 < In::kStages ? stage + 1 : 0;
    }
    if (open && e <= reach) run_out();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const long long i = ((long long)tile * a.C + c + v) * (W + 1);
        if (!in_range(i, W + 1, (long long)a.tiles * a.C * (W + 1), a.pack.status)) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) a.part[i + j] = dw[j][v];
        a.part[i + W] = db[v];
    }
}

// One thread for V channels of `rows` rows, one after another (its weights are read once, the next
// row's state while this one is computed); a row's entries of the slot lie together, (W - 1) V of them.
// 256 rows of 8192 channels take 10.6 us (15.5 cold), half of it the launch and a row's latency (floor 4.6; blocks
// of three rows in two waves 13.7 and 17.6).
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(const __grid_constant__ ConvArgs a, int across, int rows) {
    const int c = ((int)(blockIdx.x % across) * kThreads + (int)threadIdx.x) * V;
    if (c >= a.C) return;
    T *y = static_cast<T *>(a.y), *pool = static_cast<T *>(a.s1);
    const long long extent = (long long)a.pack.T * a.C, n = (long long)a.slots.num_slots * a.C * (W - 1);
    const int b0 = (int)(blockIdx.x / across) * rows, b1 = min(b0 + rows, a.pack.T);
    const Channels<T, V, W> ch(a, c);
    struct Row {
        int slot;
        Vec<T, V> x, old[W - 1];
    };
    auto entry_at = [&](int slot) { return ((long long)slot * a.C + c) * (W - 1); };
    auto read = [&](int b, Row &r) {
        r.slot = slot_of(a.slots, b);
        if (r.slot < 0) return;
        r.x = ch.token(a.x, b, a.x_stride);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) r.old[k] = load_vec<V>(pool, entry_at(r.slot) + k * V, n, a.pack.status);
    };
    Row row, next;
    read(b0, row);
    for (int b = b0; b < b1; ++b) {
        // (no two active rows have one slot: what the next row reads this one does not write)
        if (b + 1 < b1) read(b + 1, next);
        Vec<T, V> out;
        if (row.slot < 0) {
            if (c == 0 && a.slots.status && a.slots.idx[b] >= a.slots.num_slots) *a.slots.status = 1;
#pragma unroll
            for (int v = 0; v < V; ++v) out.x[v] = as_type<T>(0.f);
        } else {
            auto entry = [&](int at) { return row.old[at / V].x[at % V]; };
            Vec<T, V> now[W - 1];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float u = fmaf(ch.w[W - 1][v], as_float(row.x.x[v]), ch.b[v]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) u = fmaf(ch.w[j][v], as_float(entry(v * (W - 1) + j)), u);
                out.x[v] = as_type<T>(a.silu ? u * sigmoid_of(u) : u);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const int at = v * (W - 1) + j;
                    now[at / V].x[at % V] = j + 1 < W - 1 ? entry(at + 1) : row.x.x[v];
                }
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k) store_vec<V>(pool, entry_at(row.slot) + k * V, n, a.pack.status, now[k]);
        }
        store_vec<V>(y, (long long)b * a.C + c, extent, a.pack.status, out);
        row = next;
    }
}

// Block of 32 columns and 32 groups of rows: group g adds rows g, g + 32, ...; then the groups in order.
constexpr int kFoldGroups = 32;
__global__ void __launch_bounds__(32 * kFoldGroups) k_fold(const __grid_constant__ FoldArgs a) {
    __shared__ float sums[kFoldGroups][33];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const long long col = (long long)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (col < a.cols && in_range(col, 1, a.cols, nullptr)) {
        const float *p = a.part + col;
#pragma unroll 4
        for (long long r = group; r < a.rows; r += kFoldGroups) sum += p[r * a.cols];
    }
    sums[group][lane] = sum;
    __syncthreads();
    if (group || col >= a.cols) return;
#pragma unroll
    for (int g = 1; g < kFoldGroups; ++g) sum += sums[g][lane];
    const long long at = col / a.per;
    const int k = (int)(col % a.per);
    if (k < a.keep) a.main[at * a.keep + k] = sum;
    else if (a.rest) a.rest[at * (a.per - a.keep) + k - a.keep] = sum;
}

bool fits(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// How threads are laid out over `per` threads of a tile.  Blocks of one tile each leave some idle; where that
// is more than a fifth the threads of several tiles share a block (17 channels, gradient of 2M tokens:
// 326 us, flat 148; 8191 channels of 4096 tokens 94 and 119, as a tile's numbers are no longer a block's).
struct Layout {
    long long per;
    bool flat;
    explicit Layout(long long threads) : per(threads) {
        const long long whole = (per + kThreads - 1) / kThreads * kThreads;
        flat = 4 * whole > 5 * per;
        if (!flat) per = whole;
    }
    long long blocks(long long T, int tile) const { return ((T + tile - 1) / tile * per + kThreads - 1) / kThreads; }
    // Tokens of a tile: long ones read fewer inputs twice (W - 1 of them a tile), short ones spread a
    // small call over the SMs.
    int tile(long long T, int most) const {
        int tile = most;
        while (tile > 8 && blocks(T, tile) < 8 * 152) tile /= 2;
        return tile;
    }
};

template <typename T, int W>
cudaError_t conv_fwd(ConvArgs &a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T), kBytes = 16;
    const bool wide = a.C % V == 0 && a.x_stride % V == 0 && fits(a.x, kBytes) && fits(a.y, kBytes);
    const Layout layout(wide ? a.C / V : a.C);
    a.tile = layout.tile(a.pack.T, 64);
    const long long blocks = layout.blocks(a.pack.T, a.tile);
    const long long states = (long long)a.pack.N * (wide ? state_blocks<V>(a.C) : state_blocks<1>(a.C)), ends = a.s1 ? states : 0;
    const bool pool = a.slots.idx != nullptr, check = a.pack.status != nullptr;
    // (the check's block is the one behind the blocks of all states)
    auto launch = [&](long long first, long long grid) {
        if (grid == 0) return;
        auto with = [&](auto kernel) { kernel<<<(unsigned)grid, kThreads, 0, s>>>(a, first); };
        if (wide) layout.flat ? with(k_conv_fwd<T, V, W, true>) : with(k_conv_fwd<T, V, W, false>);
        else layout.flat ? with(k_conv_fwd<T, 1, W, true>) : with(k_conv_fwd<T, 1, W, false>);
    };
    const long long behind = check ? states + 1 : ends;
    if (pool) {
        launch(blocks, blocks);
        launch(0, behind);
    } else {
        launch(blocks, blocks + behind);
    }
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t conv_bwd(ConvArgs &a, cudaStream_t s) {
    // (8 bytes of bf16 a thread: 16 would not leave the registers for its sums and windows)
    constexpr int V = 4;
    const bool wide = a.C % V == 0 && a.x_stride % V == 0 && fits(a.x, V * sizeof(T)) && fits(a.dy, V * sizeof(T)) &&
                      fits(a.dx, V * sizeof(T));
    const Layout layout(wide ? a.C / V : a.C);
    const long long blocks = layout.blocks(a.pack.T, a.tile);
    const long long states = (long long)a.pack.N * (wide ? state_blocks<V>(a.C) : state_blocks<1>(a.C));
    const long long grid = blocks + states + (a.pack.status ? 1 : 0);
    constexpr int kRing = Stream<T, 1, 2>::kStages * Stream<T, 1, 2>::kGroup * 2 * kThreads * (int)sizeof(T);   // a channel
    static_assert(kRing * V <= 64 * 1024, "three blocks an SM");
    auto with = [&](auto kernel, int bytes) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)grid, kThreads, bytes, s>>>(a, blocks);
        return cudaGetLastError();
    };
    cudaError_t e;
    if (wide) e = layout.flat ? with(k_conv_bwd<T, V, W, true>, kRing * V) : with(k_conv_bwd<T, V, W, false>, kRing * V);
    else e = layout.flat ? with(k_conv_bwd<T, 1, W, true>, kRing) : with(k_conv_bwd<T, 1, W, false>, kRing);
    if (e != cudaSuccess) return e;
    FoldArgs f{a.part, a.tiles, (long long)a.C * (W + 1), W + 1, W, a.dw, a.dbias};
    return launch_fold(f, s);
}

template <typename T, int W>
cudaError_t conv_step(const ConvArgs &a, int batch, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = a.C % V == 0 && a.x_stride % V == 0 && fits(a.x, 16) && fits(a.y, 16) && fits(a.s1, 16);
    const int vec = wide ? V : 1;
    const int across = (a.C + kThreads * vec - 1) / (kThreads * vec);
    const int rows = step_rows(batch, across, (wide ? 4 : 16) * 152);   // (what the registers leave an SM)
    const unsigned grid = (unsigned)((batch + rows - 1) / rows * (long long)across);
    if (wide) k_conv_step<T, V, W><<<grid, kThreads, 0, s>>>(a, across, rows);
    else k_conv_step<T, 1, W><<<grid, kThreads, 0, s>>>(a, across, rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fold(const FoldArgs &a, cudaStream_t s) {
    if (a.cols == 0) return cudaSuccess;
    k_fold<<<(unsigned)((a.cols + 31) / 32), 32 * kFoldGroups, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_conv_fwd(ConvArgs a, cudaStream_t s) {
    if (a.f32) return a.W == 2 ? conv_fwd<float, 2>(a, s) : a.W == 3 ? conv_fwd<float, 3>(a, s) : conv_fwd<float, 4>(a, s);
    return a.W == 2 ? conv_fwd<bf16, 2>(a, s) : a.W == 3 ? conv_fwd<bf16, 3>(a, s) : conv_fwd<bf16, 4>(a, s);
}
cudaError_t launch_conv_bwd(ConvArgs a, cudaStream_t s) {
    if (a.f32) return a.W == 2 ? conv_bwd<float, 2>(a, s) : a.W == 3 ? conv_bwd<float, 3>(a, s) : conv_bwd<float, 4>(a, s);
    return a.W == 2 ? conv_bwd<bf16, 2>(a, s) : a.W == 3 ? conv_bwd<bf16, 3>(a, s) : conv_bwd<bf16, 4>(a, s);
}
cudaError_t launch_conv_step(const ConvArgs &a, int batch, cudaStream_t s) {
    if (a.f32) return a.W == 2 ? conv_step<float, 2>(a, batch, s) : a.W == 3 ? conv_step<float, 3>(a, batch, s) : conv_step<float, 4>(a, batch, s);
    return a.W == 2 ? conv_step<bf16, 2>(a, batch, s) : a.W == 3 ? conv_step<bf16, 3>(a, batch, s) : conv_step<bf16, 4>(a, batch, s);
}

}  // namespace gdn
