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

// The gate's factor at z, and its slope: 1 - sigmoid as e^-z sigmoid where z >= 0 (a sigmoid near 1 has lost it), and
// as it stands where z < 0 (there e^-z may be infinite, and the sigmoid 0).  A NaN stays one.
__device__ __forceinline__ float gate_of(int gate, float z) {
    return sigmoid_of(z) * (gate == GDN_GATE_SIGMOID ? 1.f : z);
}
__device__ __forceinline__ float gate_of(int gate, float z, float *slope) {
    const float e = exp_of(-z), sig = reciprocal_of(1.f + e), g = sig * (gate == GDN_GATE_SIGMOID ? 1.f : z);
    *slope = fmaf(g, z < 0.f ? 1.f - sig : e * sig, gate == GDN_GATE_SIGMOID ? 0.f : sig);
    return g;
}

}  // namespace gdn
