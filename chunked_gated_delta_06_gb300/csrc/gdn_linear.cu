// gdn_linear.cu -- linear attention with a decay for each head: the sum over the value heads
// of a key head, and the single-token step (the scans are in gdn_linear_tc.cu).
#include <type_traits>

#include "gdn_linear.h"

namespace gdn {
namespace {

// dq or dk of a key head: the fp32 sums of its value heads, or of its pairs of them, added in their
// order and rounded once.  Bound by HBM: it reads 4 r bytes and writes 2 for each element (r = 3,
// 4096 tokens of 16 heads: 118 MB, which the scans before it outlast tenfold).
__global__ void k_linear_heads(const __grid_constant__ LinearArgs a, int H) {
    const LinearPass &p = a.pass[blockIdx.y];
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;  // four features of (t, h)
    const int r = p.no / H;
    if (i >= (size_t)a.T * H * (kDim / 4)) return;
    const size_t row = i / (kDim / 4), d = i % (kDim / 4) * 4;
    const float *src = p.part + row * r * kDim + d;
    if (!in_range(src - p.part, (long long)(r - 1) * kDim + 4, (long long)a.T * p.no * kDim, a.status) ||
        !in_range(row * kDim + d, 4, (long long)a.T * H * kDim, a.status))
        return;
    float4 x = *reinterpret_cast<const float4 *>(src);
    for (int j = 1; j < r; ++j) {
        const float4 y = *reinterpret_cast<const float4 *>(src + (size_t)j * kDim);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
    }
    __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p.o + row * kDim + d) =
        make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
}

constexpr int kStepWarps = 8;
constexpr int kStepRows = kDim / kStepWarps;

// One block per (row, value head), as the gated step: a warp owns 16 rows of S, a lane one
// float4 of each.  Bound by HBM, the state read and written once: 256 rows of 32 heads, 26 of
// them null, take 143 us, 6.75 TB/s or 0.99 of the measured copy rate.
// Where lam is near 1 it is a sum hi + lo: rounded to fp32 it would be off by the same 2^-25 in
// every step of a long answer.  hi is rounded towards zero and lo at least 2^-149, so that an
// infinite element of S stays infinite (inf hi + inf lo; (lam - 1) S would cancel it to NaN).
__global__ void __launch_bounds__(kStepWarps * 32)
    k_linear_step(int H, int HV, float scale, const bf16 *__restrict__ q, const bf16 *__restrict__ k,
                  const bf16 *__restrict__ v, const float *__restrict__ log_decay,
                  float *__restrict__ pool, int num_slots, const int32_t *__restrict__ idx,
                  bf16 *__restrict__ o, int32_t *status) {
    const int b = blockIdx.x / HV, hv = blockIdx.x % HV;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = idx[b];
    bf16 *orow = o + ((size_t)b * HV + hv) * kDim;
    if (slot <= 0 || slot >= num_slots) {
        if (threadIdx.x < kDim) orow[threadIdx.x] = f2bf(0.f);
        if (slot >= num_slots && threadIdx.x == 0 && status) *status = 1;
        return;
    }
    const int h = hv / (HV / H), r0 = warp * kStepRows;
    if (!in_range(((long long)slot * HV + hv) * kDim * kDim, kDim * kDim, (long long)num_slots * HV * kDim * kDim,
                  status) ||
        !in_range(((long long)b * H + h) * kDim, kDim, (long long)(gridDim.x / HV) * H * kDim, status) ||
        !in_range(orow - o, kDim, (long long)gridDim.x * kDim, status))   // (v's rows too)
        return;
    float *S = pool + ((size_t)slot * HV + hv) * kDim * kDim;
    float4 s[kStepRows];
#pragma unroll
    for (int j = 0; j < kStepRows; ++j)
        s[j] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(r0 + j) * kDim + lane * 4));
    const size_t i = ((size_t)b * H + h) * kDim + lane * 4;
    float qv[4], kv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        qv[u] = scale * bf2f(q[i + u]);
        kv[u] = bf2f(k[i + u]);
    }
    const float g = log_decay[hv];
    const bool slow = g > -0.5f;
    const float less = expm1f(g);   // lam - 1
    const float lam = slow ? __fadd_rz(1.f, less) : expf(g);
    const float lo = fmaxf(less - (lam - 1.f), __int_as_float(1));
    const bf16 *vrow = v + ((size_t)b * HV + hv) * kDim + r0;
    float mine = 0.f;
    auto rows = [&](auto near_one) {
#pragma unroll
        for (int j = 0; j < kStepRows; ++j) {
            const float vj = bf2f(vrow[j]);
            auto next = [&](float x, float k) {
                return fmaf(lam, x, near_one ? fmaf(lo, x, vj * k) : vj * k);   // (v k is exact)
            };
            s[j].x = next(s[j].x, kv[0]);
            s[j].y = next(s[j].y, kv[1]);
            s[j].z = next(s[j].z, kv[2]);
            s[j].w = next(s[j].w, kv[3]);
            __stcs(reinterpret_cast<float4 *>(S + (size_t)(r0 + j) * kDim + lane * 4), s[j]);
            const float dot = warp_sum(s[j].x * qv[0] + s[j].y * qv[1] + s[j].z * qv[2] + s[j].w * qv[3]);
            if (lane == j) mine = dot;
        }
    };
    if (slow) rows(std::true_type());
    else rows(std::false_type());
    if (lane < kStepRows) orow[r0 + lane] = f2bf(mine);
}

}  // namespace

cudaError_t launch_linear_heads(const LinearArgs &a, int H, cudaStream_t s) {
    const size_t n = (size_t)a.T * H * (kDim / 4);
    if (n == 0) return cudaSuccess;
    k_linear_heads<<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, s>>>(a, H);
    return cudaGetLastError();
}

cudaError_t launch_linear_step(int B, int H, int HV, float scale, const bf16 *q, const bf16 *k,
                               const bf16 *v, const float *log_decay, float *pool, int num_slots,
                               const int32_t *idx, bf16 *o, int32_t *status, cudaStream_t s) {
    if (B == 0) return cudaSuccess;
    k_linear_step<<<(unsigned)((size_t)B * HV), kStepWarps * 32, 0, s>>>(
        H, HV, scale, q, k, v, log_decay, pool, num_slots, idx, o, status);
    return cudaGetLastError();
}

}  // namespace gdn
