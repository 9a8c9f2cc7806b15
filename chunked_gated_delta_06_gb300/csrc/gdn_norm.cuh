// gdn_norm.cuh -- what the norm's forward and backward share: rows spread over threads.
//
// A row of D elements is D / V vectors; TPR threads take VPT of them each, so that a row is read
// once and stays in registers between its sums and its outputs.  Up to 32 threads a row the sums
// are shuffles and a block has several rows, beyond that a row is a block's.
#pragma once

#include "gdn_mixer.cuh"

namespace gdn {

template <int TPR>
constexpr int norm_threads() { return TPR <= 32 ? 256 : TPR; }

// Sums of N values over the TPR threads of a row; every thread gets them.  `turn` alternates
// between a block's rows, so that one barrier a row is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int turn) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (TPR <= 32) return;
    __shared__ float sums[2][N][TPR / 32 > 0 ? TPR / 32 : 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) sums[turn & 1][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = lane < TPR / 32 ? sums[turn & 1][i][lane] : 0.f;
#pragma unroll
        for (int o = TPR / 64; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[i] = __shfl_sync(0xffffffffu, s, 0);
    }
}

// The gate's factor and its slope at z.
__device__ __forceinline__ float gate_of(int gate, float z, float *slope) {
    const float e = exp_of(-z), sig = reciprocal_of(1.f + e);
    const float rest = z > 0.f ? e * sig : 1.f - sig;   // 1 - sig, which a sig near 1 has lost
    if (gate == GDN_GATE_SIGMOID) {
        if (slope) *slope = sig * rest;
        return sig;
    }
    if (slope) *slope = fmaf(z * sig, rest, sig);
    return z * sig;
}

// Picks threads a row and vectors a thread for nv vectors: as many threads as there are vectors, so
// that no register array is longer than it has to be, up to 512.
template <bool kWide, typename F>
cudaError_t norm_shape(int nv, F launch) {
    if constexpr (kWide) {
        if (nv <= 16) return launch.template operator()<16, 1>();
        if (nv <= 32) return launch.template operator()<32, 1>();
        if (nv <= 128) return launch.template operator()<128, 1>();
        if (nv <= 256) return launch.template operator()<256, 1>();
        if (nv <= 512) return launch.template operator()<512, 1>();
        if (nv <= 1024) return launch.template operator()<256, 4>();
        return launch.template operator()<512, 4>();
    } else {
        if (nv <= 128) return launch.template operator()<128, 1>();
        if (nv <= 2048) return launch.template operator()<512, 4>();
        return launch.template operator()<1024, 8>();
    }
}

}  // namespace gdn
