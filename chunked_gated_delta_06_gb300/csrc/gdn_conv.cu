// gdn_conv.cu -- the short causal convolution of packed sequences: forward (also over pool slots),
// backward and a step of one token for each row.
//
// Channel c of token t, with W weights and what came before the sequence in its state:
//   u_t = bias + sum_j w_j x_{t-(W-1)+j},   y_t = u_t or u_t sigmoid(u_t)
// and with d_t = dy_t y'(u_t):
//   dx_t = sum_j w_j d_{t+(W-1)-j},   dw_j = sum_t d_t x_{t-(W-1)+j},   dbias = sum_t d_t
// The state is the last W - 1 inputs, oldest first, so it has no arithmetic of its own.
#include <algorithm>

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
                const Vec<T, V> x = token(a.x, p, a.x_stride);
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = as_float(x.x[v]);
            } else {
                state(a.s0, row, rows(), p - s + W - 1, win[k]);
            }
        }
    }
    __device__ float pre(const float (&win)[W][V], int v) const {
        float u = b[v];
#pragma unroll
        for (int j = 0; j < W; ++j) u = fmaf(w[j][v], win[j][v], u);
        return u;
    }
    __device__ static void shift(float (&win)[W][V]) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
    }
};

// The state behind sequence n: its last W - 1 inputs, the older ones from the state ahead of it.
// The thread that reads a channel's old state writes the new one, so a slot may hold both.
template <typename T, int W>
__device__ void final_state(const ConvArgs &a, int n, int c) {
    if (c >= a.C || !a.s1) return;
    const int s = offset_of(a.pack, n), e = max(s, offset_of(a.pack, n + 1));
    const int row = start_row(a, n), to = a.slots.idx ? slot_of(a.slots, n) : n;
    const Channels<T, 1, W> ch(a, c);
    if (a.slots.idx && c == 0 && a.slots.status && a.slots.idx[n] >= a.slots.num_slots) *a.slots.status = 1;
    if (to < 0) return;
    float out[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int p = e - (W - 1) + k;
        float x[1];
        if (p >= s) x[0] = as_float(ch.token(a.x, p, a.x_stride).x[0]);
        else ch.state(a.s0, row, ch.rows(), p - s + W - 1, x);
        out[k] = x[0];
    }
    const long long i = ((long long)to * a.C + c) * (W - 1);
    if (in_range(i, W - 1, (long long)ch.rows() * a.C * (W - 1), a.pack.status))
#pragma unroll
        for (int k = 0; k < W - 1; ++k) static_cast<T *>(a.s1)[i + k] = as_type<T>(out[k]);
}

// A thread walks the tokens of a tile for V channels with the last W - 1 inputs in registers, U
// tokens' loads at once.  The blocks behind those of the tiles write the states behind the
// sequences (over a pool they are a launch of their own: the tiles still read the slots).
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_fwd(const __grid_constant__ ConvArgs a, int across, long long blocks) {
    constexpr int U = 8;
    const long long block = blockIdx.x;
    if (block >= blocks) {
        const int per = (a.C + kThreads - 1) / kThreads;
        const long long i = block - blocks;
        if (i >= (long long)a.pack.N * per) check_offsets(a.pack);
        else final_state<T, W>(a, (int)(i / per), (int)(i % per) * kThreads + (int)threadIdx.x);
        return;
    }
    const int c = ((int)(block % across) * kThreads + (int)threadIdx.x) * V;
    if (c >= a.C) return;
    const int t0 = (int)(block / across) * a.tile, t1 = (int)min((long long)t0 + a.tile, (long long)a.pack.T);
    const Channels<T, V, W> ch(a, c);
    T *y = static_cast<T *>(a.y);
    const long long extent = (long long)a.pack.T * a.C;
    for (int t = t0; t < t1;) {
        const int n = sequence_of(a.pack, t), s = min(offset_of(a.pack, n), t);
        int end = offset_of(a.pack, n + 1);
        end = end > t ? min(end, t1) : t1;
        float win[W][V];
        ch.window(n, s, t, win);
        auto one = [&](const Vec<T, V> &x) {
            Vec<T, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                win[W - 1][v] = as_float(x.x[v]);
                const float u = ch.pre(win, v);
                out.x[v] = as_type<T>(a.silu ? u * sigmoid_of(u) : u);
            }
            ch.shift(win);
            store_vec<V>(y, (long long)t * a.C + c, extent, a.pack.status, out);
            ++t;
        };
        for (; t + U <= end;) {
            Vec<T, V> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = ch.token(a.x, t + u, a.x_stride);
#pragma unroll
            for (int u = 0; u < U; ++u) one(x[u]);
        }
        for (; t < end;) one(ch.token(a.x, t, a.x_stride));
    }
}

// A thread walks a tile and the W - 1 tokens behind it: at token t it has d_t and, with the d's
// before, dx of token t - (W - 1) (where that lies ahead of the sequence, of its state's entry).
// Sums for dw and dbias are of the tile's own tokens; k_fold adds the tiles.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(const __grid_constant__ ConvArgs a, int across, long long blocks) {
    constexpr int U = 4;
    const long long block = blockIdx.x;
    if (block >= blocks) {   // sequences without tokens: the state passed through
        const int per = (a.C + kThreads - 1) / kThreads;
        const long long i = block - blocks;
        if (i >= (long long)a.pack.N * per) {
            check_offsets(a.pack);
            return;
        }
        const int n = (int)(i / per), c = (int)(i % per) * kThreads + (int)threadIdx.x;
        if (c >= a.C || !a.ds0 || offset_of(a.pack, n + 1) > offset_of(a.pack, n)) return;
        const long long at = ((long long)n * a.C + c) * (W - 1);
        if (!in_range(at, W - 1, (long long)a.pack.N * a.C * (W - 1), a.pack.status)) return;
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            static_cast<T *>(a.ds0)[at + k] = a.ds1 ? static_cast<const T *>(a.ds1)[at + k] : as_type<T>(0.f);
        return;
    }
    const int c = ((int)(block % across) * kThreads + (int)threadIdx.x) * V;
    if (c >= a.C) return;
    const int tile = (int)(block / across);
    const int t0 = tile * a.tile, t1 = (int)min((long long)t0 + a.tile, (long long)a.pack.T);
    const Channels<T, V, W> ch(a, c);
    T *dx = static_cast<T *>(a.dx);
    const long long extent = (long long)a.pack.T * a.C;
    float dw[W][V] = {}, db[V] = {};
    for (int p = t0; p < t1;) {
        const int n = sequence_of(a.pack, p), s = min(offset_of(a.pack, n), p);
        int e = offset_of(a.pack, n + 1);
        e = e > p ? e : t1;
        const int q = min(e, t1);
        float win[W][V], d[W][V] = {};   // d[k] = d_{t-(W-1)+k}
        ch.window(n, s, p, win);
        auto slope = [&](const Vec<T, V> &x, const Vec<T, V> &dy) {   // d_t, with x_t in the window
#pragma unroll
            for (int v = 0; v < V; ++v) {
                win[W - 1][v] = as_float(x.x[v]);
                d[W - 1][v] = as_float(dy.x[v]);
                if (a.silu) {
                    const float u = ch.pre(win, v), sig = sigmoid_of(u);
                    d[W - 1][v] *= fmaf(u * sig, 1.f - sig, sig);
                }
            }
        };
        auto sums = [&] {
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][v] = fmaf(d[W - 1][v], win[j][v], dw[j][v]);
                db[v] += d[W - 1][v];
            }
        };
        auto gradient = [&](int v) {
            float g = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) g = fmaf(ch.w[j][v], d[W - 1 - j][v], g);
            return g;
        };
        for (int t = p; t < q + W - 1;) {
            // in the middle: every token of the group has its own dx, none of them reaches the state
            if (t - (W - 1) >= p && t + U <= q) {
                Vec<T, V> x[U], dy[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[u] = ch.token(a.x, t + u, a.x_stride);
                    dy[u] = ch.token(a.dy, t + u, a.C);
                }
#pragma unroll
                for (int u = 0; u < U; ++u, ++t) {
                    slope(x[u], dy[u]);
                    sums();
                    Vec<T, V> out;
#pragma unroll
                    for (int v = 0; v < V; ++v) out.x[v] = as_type<T>(gradient(v));
                    store_vec<V>(dx, (long long)(t - (W - 1)) * a.C + c, extent, a.pack.status, out);
                    ch.shift(win);
                    ch.shift(d);
                }
                continue;
            }
            if (t < e && t < a.pack.T) {
                slope(ch.token(a.x, t, a.x_stride), ch.token(a.dy, t, a.C));
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) d[W - 1][v] = 0.f;
            }
            if (t < q) sums();
            const int at = t - (W - 1);
            if (at >= p || p == s) {
                // the final state's gradient: entry k holds input e - (W - 1) + k
                float tail[V] = {};
                if (a.ds1 && at >= e - (W - 1)) ch.state(a.ds1, n, a.pack.N, at - e + W - 1, tail);
                Vec<T, V> out;
#pragma unroll
                for (int v = 0; v < V; ++v) out.x[v] = as_type<T>(gradient(v) + tail[v]);
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
            }
            ch.shift(win);
            ch.shift(d);
            ++t;
        }
        p = q;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const long long i = ((long long)tile * a.C + c + v) * (W + 1);
        if (!in_range(i, W + 1, (long long)a.tiles * a.C * (W + 1), a.pack.status)) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) a.part[i + j] = dw[j][v];
        a.part[i + W] = db[v];
    }
}

// One thread for V channels of a row; their entries of the slot lie together, (W - 1) V of them.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(const __grid_constant__ ConvArgs a, int across) {
    const int b = blockIdx.x / across;
    const int c = ((int)(blockIdx.x % across) * kThreads + (int)threadIdx.x) * V;
    if (c >= a.C) return;
    const int slot = slot_of(a.slots, b);
    T *y = static_cast<T *>(a.y);
    const long long extent = (long long)a.pack.T * a.C;
    Vec<T, V> out;
    if (slot < 0) {
        if (c == 0 && a.slots.status && a.slots.idx[b] >= a.slots.num_slots) *a.slots.status = 1;
#pragma unroll
        for (int v = 0; v < V; ++v) out.x[v] = as_type<T>(0.f);
        store_vec<V>(y, (long long)b * a.C + c, extent, a.pack.status, out);
        return;
    }
    using Rows = Vec<T, V>;
    const long long i = ((long long)slot * a.C + c) * (W - 1), n = (long long)a.slots.num_slots * a.C * (W - 1);
    T *pool = static_cast<T *>(a.s1);
    const Channels<T, V, W> ch(a, c);
    const Vec<T, V> x = ch.token(a.x, b, a.x_stride);
    Rows old[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) old[k] = load_vec<V>(pool, i + k * V, n, a.pack.status);
    auto entry = [&](int at) { return old[at / V].x[at % V]; };
    Rows next[W - 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float u = fmaf(ch.w[W - 1][v], as_float(x.x[v]), ch.b[v]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) u = fmaf(ch.w[j][v], as_float(entry(v * (W - 1) + j)), u);
        out.x[v] = as_type<T>(a.silu ? u * sigmoid_of(u) : u);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int at = v * (W - 1) + j;
            next[at / V].x[at % V] = j + 1 < W - 1 ? entry(at + 1) : x.x[v];
        }
    }
    store_vec<V>(y, (long long)b * a.C + c, extent, a.pack.status, out);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<V>(pool, i + k * V, n, a.pack.status, next[k]);
}

// Block of 32 columns and 8 groups of rows: group g adds rows g, g + 8, ...; then the groups in order.
__global__ void __launch_bounds__(256) k_fold(const __grid_constant__ FoldArgs a) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const long long col = (long long)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (col < a.cols && in_range(col, 1, a.cols, nullptr)) {
        const float *p = a.part + col;
#pragma unroll 4
        for (long long r = group; r < a.rows; r += 8) sum += p[r * a.cols];
    }
    sums[group][lane] = sum;
    __syncthreads();
    if (group || col >= a.cols) return;
    for (int g = 1; g < 8; ++g) sum += sums[g][lane];
    const long long at = col / a.per;
    const int k = (int)(col % a.per);
    if (k < a.keep) a.main[at * a.keep + k] = sum;
    else if (a.rest) a.rest[at * (a.per - a.keep) + k - a.keep] = sum;
}

bool fits(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Tokens of a tile: long ones read fewer inputs twice (W - 1 of them a tile), short ones spread a
// small call over the SMs.
int tile_of(long long T, long long across, int most) {
    int tile = most;
    while (tile > 8 && (T + tile - 1) / tile * across < 8 * 152) tile /= 2;
    return tile;
}

template <typename T, int W>
cudaError_t conv_fwd(ConvArgs &a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = a.C % V == 0 && a.x_stride % V == 0 && fits(a.x, 16) && fits(a.y, 16);
    const int vec = wide ? V : 1;
    const int across = (a.C + kThreads * vec - 1) / (kThreads * vec);
    a.tile = tile_of(a.pack.T, across, 64);
    const long long blocks = ((long long)a.pack.T + a.tile - 1) / a.tile * across;
    const long long ends = a.s1 ? (long long)a.pack.N * ((a.C + kThreads - 1) / kThreads) : 0;
    const bool pool = a.slots.idx != nullptr, check = a.pack.status != nullptr;
    // (the check's block is the one behind the blocks of all states)
    auto launch = [&](long long first, long long grid) {
        if (grid == 0) return;
        if (wide) k_conv_fwd<T, V, W><<<(unsigned)grid, kThreads, 0, s>>>(a, across, first);
        else k_conv_fwd<T, 1, W><<<(unsigned)grid, kThreads, 0, s>>>(a, across, first);
    };
    const long long per = (long long)a.pack.N * ((a.C + kThreads - 1) / kThreads);
    const long long behind = check ? per + 1 : ends;
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
    const int vec = wide ? V : 1;
    const int across = (a.C + kThreads * vec - 1) / (kThreads * vec);
    const long long blocks = (long long)a.tiles * across;
    const long long grid = blocks + (long long)a.pack.N * ((a.C + kThreads - 1) / kThreads) + (a.pack.status ? 1 : 0);
    if (wide) k_conv_bwd<T, V, W><<<(unsigned)grid, kThreads, 0, s>>>(a, across, blocks);
    else k_conv_bwd<T, 1, W><<<(unsigned)grid, kThreads, 0, s>>>(a, across, blocks);
    const cudaError_t e = cudaGetLastError();
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
    const unsigned grid = (unsigned)((long long)batch * across);
    if (wide) k_conv_step<T, V, W><<<grid, kThreads, 0, s>>>(a, across);
    else k_conv_step<T, 1, W><<<grid, kThreads, 0, s>>>(a, across);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fold(const FoldArgs &a, cudaStream_t s) {
    if (a.cols == 0) return cudaSuccess;
    k_fold<<<(unsigned)((a.cols + 31) / 32), 256, 0, s>>>(a);
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
