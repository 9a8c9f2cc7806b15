// gdn_norm.cu -- the norm ahead of or behind a block, with its residual and gate:
//   h = residual + scale x, rounded to the stream's type (or h = x),
//   y = h / sqrt(mean(h^2) + eps) (offset + w) act(z)
// The norm is of h as it is stored, so that the backward sees the numbers that the forward saw.
// Bound by HBM, every element read and written once: 1M rows of 128 with a silu gate (bf16) take 130 us, 6.2 TB/s or
// 0.92 of the copy rate.  (One row a thread at a time: 203 us; two rows at once and words for pairs of bf16, 131.)
#include <type_traits>

#include "gdn_norm.cuh"

namespace gdn {
namespace {

// Picks threads a row and vectors a thread for nv vectors: as many threads as there are vectors, so
// that no register array is longer than it has to be, up to 512.  Rows that are no whole vectors go
// element by element, a warp for a row of up to 256.
template <bool kWide, typename F>
cudaError_t norm_shape(int nv, F launch) {
    if (nv <= 4) return launch.template operator()<4, 1>();
    if (nv <= 8) return launch.template operator()<8, 1>();
    if (nv <= 16) return launch.template operator()<16, 1>();
    if (nv <= 32) return launch.template operator()<32, 1>();
    if constexpr (kWide) {
        if (nv <= 128) return launch.template operator()<128, 1>();
        if (nv <= 256) return launch.template operator()<256, 1>();
        if (nv <= 512) return launch.template operator()<512, 1>();
        if (nv <= 1024) return launch.template operator()<256, 4>();
        return launch.template operator()<512, 4>();
    } else {
        if (nv <= 64) return launch.template operator()<32, 2>();
        if (nv <= 256) return launch.template operator()<32, 8>();
        if (nv <= 1024) return launch.template operator()<128, 8>();
        if (nv <= 2048) return launch.template operator()<512, 4>();
        if (nv <= 4096) return launch.template operator()<512, 8>();
        return launch.template operator()<1024, 8>();
    }
}

// Rows of a thread at once: what a thread has on its way is what keeps HBM busy.
template <int TPR, int VPT, int V>
constexpr int norm_rows() { return TPR <= 32 && V > 1 ? 2 : 1; }

// kStream: with a residual.
template <typename T, typename R, int V, int TPR, int VPT, bool kStream>
__global__ void __launch_bounds__(norm_threads<TPR>(), TPR <= 32 ? 4 : 1) k_norm_fwd(const __grid_constant__ NormArgs a) {
    constexpr int J = norm_rows<TPR, VPT, V>();
    constexpr int kRows = norm_threads<TPR>() / TPR;
    const int lane = threadIdx.x % TPR, nv = a.D / V;
    const long long extent = a.R * a.D;
    const long long r0 = (long long)blockIdx.x * kRows * J + threadIdx.x / TPR;   // its rows are kRows apart
    const long long at0 = r0 * a.D + lane * V;
    const T *x = static_cast<const T *>(a.x), *z = static_cast<const T *>(a.z);
    const R *res = static_cast<const R *>(a.residual);
    auto at = [&](int j, int k) { return at0 + (long long)(j * kRows) * a.D + k * TPR * V; };
    auto there = [&](int j, int k) { return r0 + j * kRows < a.R && lane + k * TPR < nv; };
    Vec<T, V> xv[J][VPT], zv[J][VPT];
    Vec<R, V> hv[J][VPT];
    float sums[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!there(j, k)) continue;
            xv[j][k] = load_vec<V>(x, at(j, k), extent, nullptr);
            if (z) zv[j][k] = load_vec<V>(z, at(j, k), extent, nullptr);
            if (kStream) hv[j][k] = load_vec<V>(res, at(j, k), extent, nullptr);
        }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        sums[j] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!there(j, k)) continue;
            float h[V];
            if (kStream) {
                Vec<float, V> scale;
                if (a.scale) scale = load_vec<V>(a.scale, (long long)(lane + k * TPR) * V, a.D, nullptr);
                float branch[V];
                unpack(xv[j][k], branch);
                unpack(hv[j][k], h);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] += a.scale ? scale.x[v] * branch[v] : branch[v];
                hv[j][k] = pack<R>(h);
                store_vec<V>(static_cast<R *>(a.h), at(j, k), extent, nullptr, hv[j][k]);
                unpack(hv[j][k], h);
            } else {
                unpack(xv[j][k], h);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) sums[j] = fmaf(h[v], h[v], sums[j]);
        }
    }
    row_sums<TPR>(sums, 0);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = lane + k * TPR;
        if (i >= nv) break;
        Vec<float, V> w = load_vec<V>(a.w, (long long)i * V, a.D, nullptr);
#pragma unroll
        for (int v = 0; v < V; ++v) w.x[v] += a.offset;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!there(j, k)) break;
            const float r = rsqrtf(fmaf(sums[j], a.per_d, a.eps));
            float y[V], g[V];
            if (kStream) unpack(hv[j][k], y);
            else unpack(xv[j][k], y);
            if (z) unpack(zv[j][k], g);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                y[v] *= r * w.x[v];
                if (z) y[v] *= gate_of(a.gate, g[v]);
            }
            store_vec<V>(static_cast<T *>(a.y), at(j, k), extent, nullptr, pack<T>(y));
        }
    }
}

template <typename T, typename R, int V>
struct Launch {
    const NormArgs &a;
    cudaStream_t s;
    template <int TPR, int VPT>
    cudaError_t operator()() const {
        const long long rows = norm_threads<TPR>() / TPR * norm_rows<TPR, VPT, V>();
        const unsigned grid = (unsigned)((a.R + rows - 1) / rows);
        if (a.residual) k_norm_fwd<T, R, V, TPR, VPT, true><<<grid, norm_threads<TPR>(), 0, s>>>(a);
        else if constexpr (std::is_same_v<T, R>) k_norm_fwd<T, R, V, TPR, VPT, false><<<grid, norm_threads<TPR>(), 0, s>>>(a);
        return cudaGetLastError();
    }
};

template <typename T, typename R>
cudaError_t norm_fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    // (the host has checked that every tensor starts on 16 bytes)
    if (a.D % V == 0) return norm_shape<true>(a.D / V, Launch<T, R, V>{a, s});
    return norm_shape<false>(a.D, Launch<T, R, 1>{a, s});
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
    if (a.R == 0) return cudaSuccess;
    if (a.f32) return norm_fwd<float, float>(a, s);
    return a.res == GDN_DTYPE_F32 ? norm_fwd<bf16, float>(a, s) : norm_fwd<bf16, bf16>(a, s);
}

}  // namespace gdn
