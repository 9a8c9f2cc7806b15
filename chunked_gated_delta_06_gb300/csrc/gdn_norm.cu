// gdn_norm.cu -- the norm ahead of or behind a block, with its residual and gate:
//   h = residual + scale x, rounded to the stream's type (or h = x),
//   y = h / sqrt(mean(h^2) + eps) (offset + w) act(z)
// The norm is of h as it is stored, so that the backward sees the numbers that the forward saw.
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <typename T, typename R, int V, int TPR, int VPT>
__global__ void __launch_bounds__(norm_threads<TPR>()) k_norm_fwd(const __grid_constant__ NormArgs a) {
    constexpr int J = TPR <= 32 ? 2 : 1;   // rows of a thread at once
    constexpr int kRows = norm_threads<TPR>() / TPR;
    const int lane = threadIdx.x % TPR, nv = a.D / V;
    const long long extent = a.R * a.D;
    const long long r0 = ((long long)blockIdx.x * kRows + threadIdx.x / TPR) * J;
    const T *x = static_cast<const T *>(a.x), *z = static_cast<const T *>(a.z);
    Vec<T, V> zv[J][VPT];
    float h[J][VPT][V], sums[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        Vec<T, V> xv[VPT];
        Vec<R, V> rv[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            const long long at = (r0 + j) * a.D + (long long)i * V;
            if (r0 + j < a.R && i < nv) {
                xv[k] = load_vec<V>(x, at, extent, nullptr);
                if (a.z) zv[j][k] = load_vec<V>(z, at, extent, nullptr);
                if (a.residual) rv[k] = load_vec<V>(static_cast<const R *>(a.residual), at, extent, nullptr);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            const bool there = r0 + j < a.R && i < nv;
            Vec<float, V> scale;
            if (there && a.scale) scale = load_vec<V>(a.scale, (long long)i * V, a.D, nullptr);
            Vec<R, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[j][k][v] = there ? as_float(xv[k].x[v]) : 0.f;
                if (a.residual && there) {
                    const float branch = a.scale ? scale.x[v] * h[j][k][v] : h[j][k][v];
                    out.x[v] = as_type<R>(as_float(rv[k].x[v]) + branch);
                    h[j][k][v] = as_float(out.x[v]);
                }
                sum = fmaf(h[j][k][v], h[j][k][v], sum);
            }
            if (a.residual && there)
                store_vec<V>(static_cast<R *>(a.h), (r0 + j) * a.D + (long long)i * V, extent, nullptr, out);
        }
        sums[j] = sum;
    }
    row_sums<TPR>(sums, 0);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = lane + k * TPR;
        if (i >= nv) break;
        const Vec<float, V> w = load_vec<V>(a.w, (long long)i * V, a.D, nullptr);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (r0 + j >= a.R) break;
            const float r = rsqrtf(sums[j] / (float)a.D + a.eps);
            Vec<T, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float y = h[j][k][v] * r * (a.offset + w.x[v]);
                if (a.z) y *= gate_of(a.gate, as_float(zv[j][k].x[v]), nullptr);
                out.x[v] = as_type<T>(y);
            }
            store_vec<V>(static_cast<T *>(a.y), (r0 + j) * a.D + (long long)i * V, extent, nullptr, out);
        }
    }
}

template <typename T, typename R, int V>
struct Launch {
    const NormArgs &a;
    cudaStream_t s;
    template <int TPR, int VPT>
    cudaError_t operator()() const {
        const long long rows = norm_threads<TPR>() / TPR * (TPR <= 32 ? 2 : 1);
        k_norm_fwd<T, R, V, TPR, VPT><<<(unsigned)((a.R + rows - 1) / rows), norm_threads<TPR>(), 0, s>>>(a);
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
