// gdn_norm_bwd.cu -- gradient of the norm with its residual and gate (gdn_norm.cu).  With
// n = h r, r = 1 / sqrt(mean(h^2) + eps), u = dy act(z), e = u (offset + w):
//   dz = dy n (offset + w) act'(z),   dw = sum over rows of u n,
//   dh' = dh + r (e - n mean(e n)),   dresidual = dh',   dx = scale dh',   dscale = sum of dh' x
// A row is read once: mean(h^2) and mean(e h) come from one pair of sums.  A block walks rows far
// apart and keeps its sums for dw and dscale in registers; k_fold adds the blocks in their order.
// Bound by HBM: each thread's part of the next rows is on its way into shared memory, by asynchronous
// copies, while a row is computed (from registers alone a block has one row, and waits for it).
// 512K rows of 128, silu gate, bf16: 108 us, 6.2 TB/s or 0.91 of the copy rate (8-byte vectors 174 us, 456 blocks where
// 304 run at once 113).  16384 rows of 4096 with an fp32 stream and a scale: 215 us, 5.6 TB/s or 0.83, where the
// sums for dw and dscale leave two blocks of 512 threads an SM.  That is not the bytes alone: rows wider than 32
// vectors of 16 bytes have 8 elements a thread, read and gated twice, with a barrier and two chains of shuffles a
// row, 3 ps an element: of as many elements as those 512K rows, D = 512 .. 6000, gated, take 200 to 215 us, and a
// bf16 stream without a gate or a scale 148, where their bytes are 99.
#include <algorithm>
#include <type_traits>

#include "gdn_norm.cuh"

namespace gdn {
namespace {

// Threads a row and vectors (of V elements) a thread: 16 bytes of short rows, 4 elements of the others
// (whose sums for dw and dscale would take the registers of half the blocks), single elements of rows that
// are no whole vectors.
template <int E, typename F>   // E: elements of 16 bytes
cudaError_t norm_bwd_shape(int D, F launch) {
    if (D % E == 0 && D <= 4 * E) return launch.template operator()<4, 1, E>();
    if (D % E == 0 && D <= 8 * E) return launch.template operator()<8, 1, E>();
    if (D % E == 0 && D <= 16 * E) return launch.template operator()<16, 1, E>();
    if (D % E == 0 && D <= 32 * E) return launch.template operator()<32, 1, E>();
    const bool wide = D % 4 == 0;
    const int nv = wide ? D / 4 : D;
    if (wide) {
        if (nv <= 4) return launch.template operator()<4, 1, 4>();
        if (nv <= 8) return launch.template operator()<8, 1, 4>();
        if (nv <= 32) return launch.template operator()<32, 1, 4>();
        if (nv <= 128) return launch.template operator()<64, 2, 4>();
        if (nv <= 256) return launch.template operator()<128, 2, 4>();
        if (nv <= 512) return launch.template operator()<256, 2, 4>();
        if (nv <= 1024) return launch.template operator()<512, 2, 4>();
        return launch.template operator()<512, 4, 4>();
    }
    if (nv <= 4) return launch.template operator()<4, 1, 1>();
    if (nv <= 8) return launch.template operator()<8, 1, 1>();
    if (nv <= 32) return launch.template operator()<32, 1, 1>();
    if (nv <= 64) return launch.template operator()<32, 2, 1>();
    if (nv <= 256) return launch.template operator()<32, 8, 1>();
    if (nv <= 1024) return launch.template operator()<128, 8, 1>();
    if (nv <= 2048) return launch.template operator()<512, 4, 1>();
    return launch.template operator()<1024, 8, 1>();
}

// Where a thread's vectors of the tensors are in its part of a stage, in bytes.
template <typename T, typename R, int V>
struct Places {
    int h, dy, z, dh, x, all;
    __host__ __device__ Places(bool has_z, bool has_dh, bool has_x) {
        constexpr int t = V * (int)sizeof(T), r = V * (int)sizeof(R);
        h = 0;
        dy = r;
        z = dy + t;
        dh = z + (has_z ? t : 0);
        x = dh + (has_dh ? r : 0);
        all = x + (has_x ? t : 0);
    }
};

// kAhead: rows come through shared memory, norm_stages of them: the next one, where a row is a block's
// (and several blocks share an SM), three for the short ones.
template <int TPR>
constexpr int norm_stages() { return TPR <= 32 ? 4 : 2; }

// Blocks of an SM that the registers are to allow.
template <int TPR, int VPT, int V>
constexpr int norm_resident() { return TPR <= 32 ? (V * VPT > 4 ? 2 : 3) : V * VPT <= 8 ? 1024 / TPR : 1; }

template <typename T, typename R, int V, int TPR, int VPT, bool kAhead, bool kScale>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_resident<TPR, VPT, V>())
    k_norm_bwd(const __grid_constant__ NormArgs a) {
    constexpr int kThreads = norm_threads<TPR>(), kRows = kThreads / TPR, kStages = norm_stages<TPR>();
    constexpr bool kKeep = TPR <= 32;   // a row's values stay in registers over its sums
    extern __shared__ __align__(16) unsigned char ring[];   // [kStages][tensors][VPT][threads]
    const int lane = threadIdx.x % TPR, nv = a.D / V;
    const long long extent = a.R * a.D;
    const T *x = static_cast<const T *>(a.x), *z = static_cast<const T *>(a.z), *dy = static_cast<const T *>(a.dy);
    const R *hin = static_cast<const R *>(a.hin), *dh = static_cast<const R *>(a.dh);
    const Places<T, R, V> places(a.z != nullptr, a.dh != nullptr, kScale);
    float dw[VPT][V] = {}, ds[VPT][V] = {};
    int turn = 0;
    const long long step = (long long)gridDim.x * kRows, first = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    auto place = [&](int stage, int tensor, int k, int bytes) {
        return ring + (size_t)((stage * places.all + tensor) * VPT + k * bytes) * kThreads + threadIdx.x * bytes;
    };
    [[maybe_unused]] auto fetch = [&](long long r, int stage) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            const long long at = r * a.D + (long long)i * V;
            if (r >= a.R || i >= nv || !in_range(at, V, extent, nullptr)) continue;
            auto copy = [&](int tensor, const auto *p) {
                constexpr int kBytes = V * (int)sizeof(*p);
                constexpr int kEach = kBytes > 16 ? 16 : kBytes;
                static_assert(!kAhead || kEach >= 4, "single elements do not come through the ring");
#pragma unroll
                for (int b = 0; b < kBytes; b += kEach)
                    copy_async<kEach>(place(stage, tensor, k, kBytes) + b, reinterpret_cast<const char *>(p + at) + b, true);
            };
            copy(places.h, hin);
            copy(places.dy, dy);
            if (z) copy(places.z, z);
            if (dh) copy(places.dh, dh);
            if (kScale) copy(places.x, x);
        }
    };
    if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            fetch(first + i * step, i);
            copies_commit();
        }
    }
    auto weight = [&](int k, float (&w)[V]) {
        unpack(load_vec<V>(a.w, (long long)(lane + k * TPR) * V, a.D, nullptr), w);
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] += a.offset;
    };
    float kept_w[kKeep ? VPT : 1][V];
    if constexpr (kKeep)
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (lane + k * TPR < nv) weight(k, kept_w[k]);
    // (a block's rows: the same number for all of its threads)
    for (long long row = (long long)blockIdx.x * kRows, r = first; row < a.R; row += step, r += step, ++turn) {
        if constexpr (kAhead) {
            fetch(r + (kStages - 1) * step, (turn + kStages - 1) % kStages);
            copies_commit();
            copies_wait<kStages - 1>();
        }
        const int stage = turn % kStages;
        auto there = [&](int k) { return r < a.R && lane + k * TPR < nv; };
        const long long at0 = r * a.D + lane * V;
        // a vector of a tensor, from the ring or from memory
        auto get = [&](const auto *p, int tensor, int k, float (&out)[V]) {
            using E = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
            if constexpr (kAhead) unpack(*reinterpret_cast<const Vec<E, V> *>(place(stage, tensor, k, V * (int)sizeof(E))), out);
            else unpack(load_vec<V>(p, at0 + k * TPR * V, extent, nullptr), out);
        };
        float sums[2] = {};
        float h[VPT][V], u[VPT][V], slope[VPT][V];   // slope: of z, times dy; all but u to be had again
        auto read = [&](int k) {
            get(hin, places.h, k, h[k]);
            get(dy, places.dy, k, u[k]);
            if (z) {
                float zv[V];
                get(z, places.z, k, zv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s;
                    const float g = gate_of(a.gate, zv[v], &s);
                    slope[k][v] = u[k][v] * s;
                    u[k][v] *= g;
                }
            }
        };
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!there(k)) continue;
            float w[V];
            if constexpr (!kKeep) weight(k, w);
            read(k);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sums[0] = fmaf(h[k][v], h[k][v], sums[0]);
                sums[1] = fmaf(u[k][v] * (kKeep ? kept_w[k][v] : w[v]), h[k][v], sums[1]);
            }
        }
        row_sums<TPR>(sums, turn);
        const float rs = rsqrtf(fmaf(sums[0], a.per_d, a.eps)), mean = sums[1] * rs * a.per_d;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!there(k)) break;
            float w[V], scale[V], xv[V], gv[V], dx[V], dz[V];
            if constexpr (!kKeep) {   // (a second time from where they are, for the blocks that the registers allow)
                weight(k, w);
                read(k);
            }
            if (kScale) unpack(load_vec<V>(a.scale, (long long)(lane + k * TPR) * V, a.D, nullptr), scale);
            if (dh) get(dh, places.dh, k, gv);
            if (kScale) get(x, places.x, k, xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = h[k][v] * rs, wv = kKeep ? kept_w[k][v] : w[v];
                if (z) dz[v] = slope[k][v] * (n * wv);
                dw[k][v] = fmaf(u[k][v], n, dw[k][v]);
                float d = rs * fmaf(u[k][v], wv, -n * mean);
                if (dh) d += gv[v];
                gv[v] = d;
                if (kScale) ds[k][v] = fmaf(d, xv[v], ds[k][v]);
                dx[v] = kScale ? d * scale[v] : d;
            }
            const long long at = at0 + k * TPR * V;
            store_vec<V>(static_cast<T *>(a.dx), at, extent, nullptr, pack<T>(dx));
            if (a.dres) store_vec<V>(static_cast<R *>(a.dres), at, extent, nullptr, pack<R>(gv));
            if (z) store_vec<V>(static_cast<T *>(a.dz), at, extent, nullptr, pack<T>(dz));
        }
    }
    // the block's rows, in order
    constexpr int parts = kScale ? 2 : 1;
    const long long n = (long long)gridDim.x * parts * a.D;
    if constexpr (kRows > 1) {
        __shared__ float all[kRows][TPR * VPT * V];
        for (int part = 0; part < parts; ++part) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    all[threadIdx.x / TPR][(lane + k * TPR) * V + v] = part ? ds[k][v] : dw[k][v];
            __syncthreads();
            for (int i = threadIdx.x; i < a.D; i += kThreads) {
                float s = 0.f;
#pragma unroll
                for (int g = 0; g < kRows; ++g) s += all[g][i];
                const long long at = ((long long)blockIdx.x * parts + part) * a.D + i;
                if (in_range(at, 1, n, nullptr)) a.part[at] = s;
            }
        }
    } else {
        for (int part = 0; part < parts; ++part)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = lane + k * TPR;
                if (i >= nv) break;
                Vec<float, V> out;
#pragma unroll
                for (int v = 0; v < V; ++v) out.x[v] = part ? ds[k][v] : dw[k][v];
                store_vec<V>(a.part, ((long long)blockIdx.x * parts + part) * a.D + (long long)i * V, n, nullptr, out);
            }
    }
}

template <typename T, typename R>
struct Launch {
    const NormArgs &a;
    cudaStream_t s;
    template <int TPR, int VPT, int V>
    cudaError_t operator()() const {
        return a.scale ? kernel<TPR, VPT, V, true>() : kernel<TPR, VPT, V, false>();
    }
    template <int TPR, int VPT, int V, bool kScale>
    cudaError_t kernel() const {
        constexpr int kThreads = norm_threads<TPR>();
        const int blocks = norm_bwd_blocks(a.R, a.D, sizeof(T) == 4);
        if constexpr (V > 1) {
            const Places<T, R, V> places(a.z != nullptr, a.dh != nullptr, a.dscale != nullptr);
            const int bytes = norm_stages<TPR>() * places.all * VPT * kThreads;
            if (bytes <= 160 * 1024) {   // (wider rows are long enough to keep loads on their way by themselves)
                const cudaError_t e = cudaFuncSetAttribute(k_norm_bwd<T, R, V, TPR, VPT, true, kScale>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
                if (e != cudaSuccess) return e;
                k_norm_bwd<T, R, V, TPR, VPT, true, kScale><<<blocks, kThreads, bytes, s>>>(a);
                return cudaGetLastError();
            }
        }
        k_norm_bwd<T, R, V, TPR, VPT, false, kScale><<<blocks, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
};

template <typename T, typename R>
cudaError_t norm_bwd(const NormArgs &a, cudaStream_t s) {
    return norm_bwd_shape<16 / (int)sizeof(T)>(a.D, Launch<T, R>{a, s});
}

struct RowsOf {
    int *out;
    template <int TPR, int VPT, int V>
    cudaError_t operator()() const {
        out[0] = norm_threads<TPR>() / TPR;
        out[1] = norm_resident<TPR, VPT, V>();
        return cudaSuccess;
    }
};

}  // namespace

// A block's sums stay in registers over its rows: as many blocks as run at once, no more.
int norm_bwd_blocks(long long R, int D, int f32) {
    int shape[2];
    if (f32) norm_bwd_shape<4>(D, RowsOf{shape});
    else norm_bwd_shape<8>(D, RowsOf{shape});
    return (int)std::max(1LL, std::min((R + shape[0] - 1) / shape[0], 152LL * shape[1]));
}

cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t s) {
    cudaError_t e;
    if (a.f32) e = norm_bwd<float, float>(a, s);
    else e = a.res == GDN_DTYPE_F32 ? norm_bwd<bf16, float>(a, s) : norm_bwd<bf16, bf16>(a, s);
    if (e != cudaSuccess) return e;
    const int parts = a.dscale ? 2 : 1, D = a.D;
    return launch_fold(FoldArgs{a.part, norm_bwd_blocks(a.R, D, a.f32), (long long)parts * D, parts * D, D, a.dw, a.dscale}, s);
}

}  // namespace gdn
