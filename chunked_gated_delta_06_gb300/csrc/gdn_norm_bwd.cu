// gdn_norm_bwd.cu -- gradient of the norm with its residual and gate (gdn_norm.cu).  With
// n = h r, r = 1 / sqrt(mean(h^2) + eps), u = dy act(z), e = u (offset + w):
//   dz = dy n (offset + w) act'(z),   dw = sum over rows of u n,
//   dh' = dh + r (e - n mean(e n)),   dresidual = dh',   dx = scale dh',   dscale = sum of dh' x
// A row is read once: mean(h^2) and mean(e h) come from one pair of sums.  A block walks rows far
// apart and keeps its sums for dw and dscale in registers; k_fold adds the blocks in their order.
#include <algorithm>

#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <typename T, typename R, int V, int TPR, int VPT>
__global__ void __launch_bounds__(norm_threads<TPR>()) k_norm_bwd(const __grid_constant__ NormArgs a) {
    constexpr int kThreads = norm_threads<TPR>(), kRows = kThreads / TPR;
    const int lane = threadIdx.x % TPR, nv = a.D / V;
    const long long extent = a.R * a.D;
    const T *x = static_cast<const T *>(a.x), *z = static_cast<const T *>(a.z), *dy = static_cast<const T *>(a.dy);
    const R *hin = static_cast<const R *>(a.hin), *dh = static_cast<const R *>(a.dh);
    float dw[VPT][V] = {}, ds[VPT][V] = {};
    int turn = 0;
    for (long long row = (long long)blockIdx.x * kRows; row < a.R; row += (long long)gridDim.x * kRows, ++turn) {
        const long long r = row + threadIdx.x / TPR;
        Vec<R, V> hv[VPT], gv[VPT];
        Vec<T, V> yv[VPT], zv[VPT], xv[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            const long long at = r * a.D + (long long)i * V;
            if (r < a.R && i < nv) {
                hv[k] = load_vec<V>(hin, at, extent, nullptr);
                yv[k] = load_vec<V>(dy, at, extent, nullptr);
                if (a.z) zv[k] = load_vec<V>(z, at, extent, nullptr);
                if (a.dh) gv[k] = load_vec<V>(dh, at, extent, nullptr);
                if (a.dscale) xv[k] = load_vec<V>(x, at, extent, nullptr);
            }
        }
        float sums[2] = {}, u[VPT][V];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            if (r >= a.R || i >= nv) {
#pragma unroll
                for (int v = 0; v < V; ++v) u[k][v] = 0.f;
                continue;
            }
            const Vec<float, V> w = load_vec<V>(a.w, (long long)i * V, a.D, nullptr);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float h = as_float(hv[k].x[v]);
                u[k][v] = as_float(yv[k].x[v]);
                if (a.z) u[k][v] *= gate_of(a.gate, as_float(zv[k].x[v]), nullptr);
                sums[0] = fmaf(h, h, sums[0]);
                sums[1] = fmaf(u[k][v] * (a.offset + w.x[v]), h, sums[1]);
            }
        }
        row_sums<TPR>(sums, turn);
        const float rs = rsqrtf(sums[0] / (float)a.D + a.eps), mean = sums[1] * rs / (float)a.D;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = lane + k * TPR;
            if (r >= a.R || i >= nv) break;
            const long long at = r * a.D + (long long)i * V;
            const Vec<float, V> w = load_vec<V>(a.w, (long long)i * V, a.D, nullptr);
            Vec<float, V> scale;
            if (a.scale) scale = load_vec<V>(a.scale, (long long)i * V, a.D, nullptr);
            Vec<T, V> dx, dz;
            Vec<R, V> dres;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = as_float(hv[k].x[v]) * rs, wv = a.offset + w.x[v];
                if (a.z) {
                    float slope;
                    gate_of(a.gate, as_float(zv[k].x[v]), &slope);
                    dz.x[v] = as_type<T>(as_float(yv[k].x[v]) * n * wv * slope);
                }
                dw[k][v] = fmaf(u[k][v], n, dw[k][v]);
                float d = rs * (u[k][v] * wv - n * mean);
                if (a.dh) d += as_float(gv[k].x[v]);
                dres.x[v] = as_type<R>(d);
                if (a.dscale) ds[k][v] = fmaf(d, as_float(xv[k].x[v]), ds[k][v]);
                dx.x[v] = as_type<T>(a.scale ? d * scale.x[v] : d);
            }
            store_vec<V>(static_cast<T *>(a.dx), at, extent, nullptr, dx);
            if (a.dres) store_vec<V>(static_cast<R *>(a.dres), at, extent, nullptr, dres);
            if (a.z) store_vec<V>(static_cast<T *>(a.dz), at, extent, nullptr, dz);
        }
    }
    // the block's rows, in order
    const int parts = a.dscale ? 2 : 1;
    const long long n = (long long)gridDim.x * parts * a.D;
    if constexpr (kRows > 1) {
        __shared__ float all[kRows][TPR * V];
        for (int part = 0; part < parts; ++part) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) all[threadIdx.x / TPR][lane * V + v] = part ? ds[0][v] : dw[0][v];
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

template <typename T, typename R, int V>
struct Launch {
    const NormArgs &a;
    cudaStream_t s;
    template <int TPR, int VPT>
    cudaError_t operator()() const {
        static_assert(TPR > 32 || VPT == 1, "the sum over a block's rows takes one vector a thread");
        k_norm_bwd<T, R, V, TPR, VPT><<<norm_bwd_blocks(a.R, a.D, a.f32), norm_threads<TPR>(), 0, s>>>(a);
        return cudaGetLastError();
    }
};

template <typename T, typename R>
cudaError_t norm_bwd(const NormArgs &a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (a.D % V == 0) return norm_shape<true>(a.D / V, Launch<T, R, V>{a, s});
    return norm_shape<false>(a.D, Launch<T, R, 1>{a, s});
}

struct RowsOf {
    int *out;
    template <int TPR, int VPT>
    cudaError_t operator()() const {
        out[0] = norm_threads<TPR>() / TPR;
        out[1] = norm_threads<TPR>();
        return cudaSuccess;
    }
};

}  // namespace

// A block's sums stay in registers over its rows: as many blocks as run at once, no more.
int norm_bwd_blocks(long long R, int D, int f32) {
    const int V = f32 ? 4 : 8;
    int shape[2];
    if (D % V == 0) norm_shape<true>(D / V, RowsOf{shape});
    else norm_shape<false>(D, RowsOf{shape});
    return (int)std::max(1LL, std::min((R + shape[0] - 1) / shape[0], 152LL * (1024 / shape[1])));
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
