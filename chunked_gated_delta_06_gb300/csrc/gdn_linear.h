// gdn_linear.h -- internal interface of the decay-only linear attention kernels.
#pragma once

#include "gdn_kernels.h"

namespace gdn {

constexpr int kLinearOrder = 128;   // packs of at most this many sequences start the longest first

// One scan of linear attention over packed sequences, for value head hv with decay
// lam = e^{log_decay[hv]} (rows r = feature of v, columns c = feature of q and k):
//   forward:  S <- lam S + w v_t k_t^T,  o_t = so S q_t           (t ascending)
//   reverse:  S <- S + w v_t k_t^T,  o_t = so S q_t,  S <- lam S  (t descending)
// The forward call is one such scan; the backward is three of them with the roles of the
// tensors exchanged.  With S the state (rows: v, columns: k) and dS the gradient of the state
// after token t (dS_t = lam dS_{t+1} + scale do_t q_t^T):
//   dq_t = scale S_t^T do_t     forward scan, (q, k, v) <- (do, v, k), state transposed
//   dk_t = dS_t^T v_t           reverse scan, (q, k, v) <- (v, do, q), w = scale, transposed
//   dv_t = dS_t k_t             reverse scan, (q, k, v) <- (k, q, do), w = scale
// and dh0 is the state that either reverse scan ends with.
// A role tensor with n heads is read at head hv / (HV / n).
struct LinearPass {
    const bf16 *q, *k, *v;    // [T, nq | nk | nv, 128]
    int nq, nk, nv;
    bf16 *o;                  // [T, no, 128], or null
    float *part;              // [T, no, 128]: fp32 outputs instead of o (summed by launch_linear_heads)
    int no;                   // output heads: HV, or HV / 2 with pair
    int pair;                 // value heads 2 x and 2 x + 1 are summed into output head x
    const float *s0;          // [N, HV, 128, 128] or null (zeros)
    float *s1;                // the same shape, or null
    int rows;                 // s0, s1 and the pool's slots hold S row by row (else column by column)
    float *seg_state;         // split scans: [items, HV, 128, 128] states after each inner segment,
    int seg_rows;             // row by row, or column by column (another scan's transposed states)
    float so, w;              // output and update factors
};
// An offset's part of a sum (mod 2^64) that holds the device's cu_seqlens against the host's: times
// an odd number of its place, so that one changed offset always changes the sum, and several but
// for a chance of 2^-64.
__host__ __device__ inline uint64_t offset_term(int i, int32_t x) {
    uint64_t m = (uint64_t)(i + 1) * 0x9e3779b97f4a7c15ull;   // 2^64 / golden ratio
    m ^= m >> 32;
    m *= 0xd1342543de82ef95ull;
    m ^= m >> 29;
    return (uint64_t)(uint32_t)x * (m | 1);
}

struct LinearArgs {
    int N, T, HV;
    int longest;              // tokens of the longest sequence (host copy of cu_seqlens)
    const float *log_decay;   // [HV]
    LinearPass pass[3];       // a forward's one scan; a backward's dq, dk, dv
    int passes, state_passes; // 1 and 1, or 3 and 2 (dk starts its segments from dv's states)
    float *pool;              // [num_slots, HV, V, K] in place of s0 / s1 (paged prefill), or null
    int num_slots;
    const int *pool_idx, *pool_resume;
    int *pool_status;
    const int *cu_dev;        // [N + 1]
    uint64_t cu_sum;          // N > kLinearOrder: the sum of the host's offset_terms
    int *status;
    // Work items: (sequence, segment), grid order.  seg_chunks > 0 (N <= kLinearOrder only) cuts
    // the sequences into segments of that many chunks, which are walked at once.
    int items, seg_chunks;
    uint16_t order[kLinearOrder];  // N <= kLinearOrder: sequences by decreasing length,
    int seg_first[kLinearOrder + 1];  // the first item of each, in that order,
    int cu[kLinearOrder + 1];      // and the host's cu_seqlens
};

cudaError_t launch_linear_tc(const LinearArgs &a, cudaStream_t s);
// dq and dk from the scans' fp32 outputs: out[t][h] = sum of part[t][x] over the no / H heads x
// of key head h, in order, as bf16 (passes 0 and 1 of a).
cudaError_t launch_linear_heads(const LinearArgs &a, int H, cudaStream_t s);

cudaError_t launch_linear_step(int B, int H, int HV, float scale, const bf16 *q, const bf16 *k,
                               const bf16 *v, const float *log_decay, float *pool, int num_slots,
                               const int32_t *idx, bf16 *o, int32_t *status, cudaStream_t s);

// Rotary positions: x1' = m (x1 c - x2 s), x2' = m (x2 c + x1 s) for the pairs of the first
// `rot` elements of every head, c + i s = e^{2 pi i pos f}.
struct RopeArgs {
    int T, Hq, Hk, D, rot;
    int interleaved, backward;
    float mscale;
    const bf16 *q, *k;
    const int32_t *pos;       // [T]
    const float *freq;        // [2, rot / 2]: turns per position, head and tail
    bf16 *qo, *ko;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s);

}  // namespace gdn
