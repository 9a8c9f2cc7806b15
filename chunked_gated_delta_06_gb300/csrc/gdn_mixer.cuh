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

// All of a vector's elements as floats, and back, each rounded once.  (bf16 in words: a shift or a mask an
// element, one conversion a pair; element by element the halves are taken apart and put together too.)
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V> &v, float (&f)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 p = bf2_to_f2(reinterpret_cast<const uint32_t *>(&v)[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = as_float(v.x[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
    Vec<T, V> v;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            reinterpret_cast<uint32_t *>(&v)[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v.x[i] = as_type<T>(f[i]);
    }
    return v;
}

// Pairs of fp32 in one instruction: the pipe takes two cycles for one, but a warp's turn is spent once.
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

// The same for vectors (element by element where they are odd): the bits are those of fmaf and of products.
template <int V>
__device__ __forceinline__ void fma_all(float (&acc)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 r = fma2(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]), make_float2(acc[v], acc[v + 1]));
            acc[v] = r.x;
            acc[v + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(a[v], b[v], acc[v]);
    }
}
template <int V>
__device__ __forceinline__ void mul_all(float (&out)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 r = mul2(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]));
            out[v] = r.x;
            out[v + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = a[v] * b[v];
    }
}

template <int V>
__device__ __forceinline__ void add_all(float (&acc)[V], const float (&a)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 r = add2(make_float2(acc[v], acc[v + 1]), make_float2(a[v], a[v + 1]));
            acc[v] = r.x;
            acc[v + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += a[v];
    }
}

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
// The same of two numbers, in packed products and sums, and of vectors.
__device__ __forceinline__ float2 exp2_of(float2 x) { return make_float2(exp2_of(x.x), exp2_of(x.y)); }
__device__ __forceinline__ float2 exp_of(float2 x) { return exp2_of(mul2(x, both(1.44269504088896341f))); }
__device__ __forceinline__ float2 reciprocal_of(float2 x) { return make_float2(reciprocal_of(x.x), reciprocal_of(x.y)); }
__device__ __forceinline__ float2 sigmoid_of(float2 x) {
    return reciprocal_of(add2(both(1.f), exp2_of(mul2(x, both(-1.44269504088896341f)))));
}
template <int V>
__device__ __forceinline__ void sigmoid_all(float (&out)[V], const float (&x)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 s = sigmoid_of(make_float2(x[v], x[v + 1]));
            out[v] = s.x;
            out[v + 1] = s.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = sigmoid_of(x[v]);
    }
}

// Asynchronous copies of `bytes` (4, 8 or 16) into shared memory; zeros instead where there is nothing.
template <int kBytes>
__device__ __forceinline__ void copy_async(void *to, const void *from, bool there) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    const int n = there ? kBytes : 0;
    if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(from), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory"); }

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
