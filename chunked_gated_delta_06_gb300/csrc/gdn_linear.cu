// gdn_linear.cu -- linear attention with a decay for each head: the token-by-token scan,
// the sum over the value heads of a key head, and the single-token step.
//
//   S_t = lam S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   lam = e^{log_decay[hv]}
// (S is V x K, the transpose of the K-major state the callers pass).  With dS the gradient
// of the state after token t (dS_t = lam dS_{t+1} + scale do_t q_t^T), the gradients are
// scans of the same form with the tensors' roles exchanged:
//   dq_t = scale S_t^T do_t     forward scan, (q, k, v) <- (do, v, k), state transposed
//   dk_t = dS_t^T v_t           reverse scan, (q, k, v) <- (v, do, q), update factor scale,
//                               state transposed
//   dv_t = dS_t k_t             reverse scan, (q, k, v) <- (k, q, do), update factor scale
// and dh0 is the state either reverse scan ends with.
#include "gdn_linear.h"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 4;                    // rows of S per warp
constexpr int kRowsPerCta = kWarps * kRows;

// Sequence n's tokens, or an empty range (flagged) when the device copy of cu_seqlens
// leaves the host's extents.
__device__ __forceinline__ void seq_range(const LinearArgs &a, int n, int &t0, int &L) {
    t0 = a.cu_dev[n];
    const int t1 = a.cu_dev[n + 1];
    L = t1 - t0;
    if (t0 < 0 || t1 < t0 || t1 > a.T || L > a.longest) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, GDN_DEVICE_CU_SEQLENS_MISMATCH);
        t0 = 0;
        L = -1;
    }
}

// Grid (N * 128 / kRowsPerCta, HV): each warp keeps kRows rows of S in registers, a lane
// four columns of each.
__global__ void __launch_bounds__(kWarps * 32) k_linear_scan(const LinearArgs a) {
    const int hv = blockIdx.y, n = blockIdx.x / (kDim / kRowsPerCta);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = blockIdx.x % (kDim / kRowsPerCta) * kRowsPerCta + warp * kRows;
    int t0, L;
    seq_range(a, n, t0, L);
    if (L < 0) return;
    const int hq = hv / (a.HV / a.nq), hk = hv / (a.HV / a.nk), hw = hv / (a.HV / a.nv);
    // lam to 48 bits: rounded to fp32, its 2^-25 would grow with every token of a slow decay
    const double lam64 = exp((double)a.log_decay[hv]);
    const float lam = (float)lam64, lam_tail = (float)(lam64 - (double)lam);
    const float *src = a.s0 ? a.s0 + ((size_t)n * a.HV + hv) * kDim * kDim : nullptr;
    float *dst = a.s1 ? a.s1 + ((size_t)n * a.HV + hv) * kDim * kDim : nullptr;
    if (a.pool) {
        const int slot = a.pool_idx[n];
        if (slot >= a.num_slots && threadIdx.x == 0 && a.pool_status) *a.pool_status = 1;
        if (slot > 0 && slot < a.num_slots) {
            dst = a.pool + ((size_t)slot * a.HV + hv) * kDim * kDim;
            src = (!a.pool_resume || a.pool_resume[n]) ? dst : nullptr;
        }
    }
    float s[kRows][4];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            s[j][u] = src ? src[(size_t)(r0 + j) * a.s_rs + (size_t)(lane * 4 + u) * a.s_cs] : 0.f;
    for (int i = 0; i < L; ++i) {
        const size_t t = (size_t)t0 + (a.reverse ? L - 1 - i : i);
        const bf16 *q = a.q + (t * a.nq + hq) * kDim + lane * 4;
        const bf16 *k = a.k + (t * a.nk + hk) * kDim + lane * 4;
        const bf16 *v = a.v + (t * a.nv + hw) * kDim + r0;
        float mine = 0.f;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const float vj = a.w * bf2f(v[j]);
            float dot = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float add = vj * bf2f(k[u]);
                if (!a.reverse) s[j][u] = fmaf(s[j][u], lam, fmaf(s[j][u], lam_tail, add));
                else s[j][u] += add;
                dot += s[j][u] * bf2f(q[u]);
                if (a.reverse) s[j][u] = fmaf(s[j][u], lam, s[j][u] * lam_tail);
            }
            dot = warp_sum(dot);
            if (lane == j) mine = a.so * dot;
        }
        if (lane < kRows) {
            const size_t i_out = (t * a.HV + hv) * kDim + r0 + lane;
            if (a.part) a.part[i_out] = mine;
            else if (a.o) a.o[i_out] = f2bf(mine);
        }
    }
    if (dst) {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                dst[(size_t)(r0 + j) * a.s_rs + (size_t)(lane * 4 + u) * a.s_cs] = s[j][u];
    }
}

__global__ void k_linear_heads(const float *__restrict__ part, bf16 *__restrict__ out, size_t rows,
                               int r, int *status) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;  // (t, h, d)
    if (i >= rows * kDim) return;
    const size_t row = i / kDim, d = i % kDim;
    if (!in_range(row * r * kDim + d, (long long)(r - 1) * kDim + 1, rows * r * kDim, status)) return;
    float x = 0.f;
    for (int j = 0; j < r; ++j) x += part[(row * r + j) * kDim + d];
    out[i] = f2bf(x);
}

constexpr int kStepWarps = 8;
constexpr int kStepRows = kDim / kStepWarps;

// One block per (row, value head), as the gated step: a warp owns 16 rows of S, a lane one
// float4 of each.
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
    const float lam = expf(log_decay[hv]);
    const bf16 *vrow = v + ((size_t)b * HV + hv) * kDim + r0;
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) {
        const float vj = bf2f(vrow[j]);
        s[j].x = lam * s[j].x + vj * kv[0];
        s[j].y = lam * s[j].y + vj * kv[1];
        s[j].z = lam * s[j].z + vj * kv[2];
        s[j].w = lam * s[j].w + vj * kv[3];
        __stcs(reinterpret_cast<float4 *>(S + (size_t)(r0 + j) * kDim + lane * 4), s[j]);
        const float dot = warp_sum(s[j].x * qv[0] + s[j].y * qv[1] + s[j].z * qv[2] + s[j].w * qv[3]);
        if (lane == j) mine = dot;
    }
    if (lane < kStepRows) orow[r0 + lane] = f2bf(mine);
}

}  // namespace

cudaError_t launch_linear_scan(const LinearArgs &a, cudaStream_t s) {
    k_linear_scan<<<dim3((unsigned)a.N * (kDim / kRowsPerCta), a.HV), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_linear_heads(const float *part, bf16 *out, int T, int H, int HV, int *status,
                                cudaStream_t s) {
    const size_t n = (size_t)T * H * kDim;
    if (n == 0) return cudaSuccess;
    k_linear_heads<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(part, out, (size_t)T * H, HV / H, status);
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
