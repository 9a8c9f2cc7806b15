// gdn_mixer.cuh -- device helpers of the convolution, scan and norm kernels.
#pragma once

#include "gdn_mixer.h"

namespace gdn {

template <typename T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Vec {
    T x[V];
};

__device__ __forceinline__ float as_float(bf16 x) { return bf2f(x); }
__device__ __forceinline__ float as_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T as_type(float x);
template <>
__device__ __forceinline__ bf16 as_type<bf16>(float x) { return f2bf(x); }
template <>
__device__ __forceinline__ float as_type<float>(float x) { return x; }

// V elements from i on of a buffer of n (zeros outside it, in the checked build).
template <int V, typename T>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p, long long i, long long n, int *status) {
    Vec<T, V> v;
    if (!in_range(i, V, n, status)) {
#pragma unroll
        for (int k = 0; k < V; ++k) v.x[k] = as_type<T>(0.f);
        return v;
    }
    return *reinterpret_cast<const Vec<T, V> *>(p + i);
}
template <int V, typename T>
__device__ __forceinline__ void store_vec(T *p, long long i, long long n, int *status, const Vec<T, V> &v) {
    if (in_range(i, V, n, status)) *reinterpret_cast<Vec<T, V> *>(p + i) = v;
}

// The hardware's 2^x and 1 / x (2^-22 each), denormal numbers taken for 0: one instruction each, where
// __expf and __fdividef keep denormals and extreme divisors for some more.
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp_of(float x) { return exp2_of(x * 1.44269504088896341f); }
__device__ __forceinline__ float reciprocal_of(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x): good to about 2^-21 for |x| < 10 (2^-24 |x| beyond), which a result in bf16 does
// not see and one in fp32 bears.
__device__ __forceinline__ float sigmoid_of(float x) { return reciprocal_of(1.f + exp_of(-x)); }

// The sequence of token t: the last n with cu[n] <= t.
__device__ __forceinline__ int sequence_of(const PackArgs &p, int t) {
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
        const int mid = (int)(((unsigned)lo + (unsigned)hi + 1) / 2);
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int offset_of(const PackArgs &p, int n) { return min(max(p.cu[n], 0), p.T); }

// One block's sum of the device's offsets against the host's.
__device__ inline void check_offsets(const PackArgs &p) {
    __shared__ unsigned long long sums[32];
    unsigned long long sum = 0;
    for (int i = threadIdx.x; i <= p.N; i += blockDim.x) sum += offset_term(i, p.cu[i]);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (unsigned w = 1; w < blockDim.x / 32; ++w) sum += sums[w];
        if (sum != p.cu_sum) atomicOr(p.status, GDN_DEVICE_CU_SEQLENS_MISMATCH);
    }
}

// The slot of sequence (or row) n, -1 for none.
__device__ __forceinline__ int slot_of(const SlotArgs &s, int n) {
    const int slot = s.idx[n];
    return slot <= 0 || slot >= s.num_slots ? -1 : slot;
}

}  // namespace gdn
