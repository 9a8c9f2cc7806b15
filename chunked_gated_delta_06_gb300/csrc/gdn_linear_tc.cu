// gdn_linear_tc.cu -- the scans of the decay-only linear attention on the tensor cores.
//
// A CTA walks the 128-token chunks of one (sequence, value head).  With i, j the positions
// of a chunk's tokens, lam the head's decay, S (rows: features of v, columns: features of q
// and k) the running state, for a forward scan
//   o_i = so ( lam^{i+1} S q_i + w sum_{j<=i} lam^{i-j} (q_i . k_j) v_j )
//   S  <- lam^L S + w sum_t lam^{L-1-t} v_t k_t^T
// and for a reverse scan (the state enters behind the chunk's last token)
//   o_i = so ( lam^{L-1-i} S q_i + w sum_{j>=i} lam^{j-i} (q_i . k_j) v_j ),
//   S  <- lam^L S + w sum_t lam^{t+1} v_t k_t^T.
//
// Products per chunk (M = N = 128, tcgen05, bf16 operands, fp32 accumulation):
//   P  = Q K^T                       both from shared memory
//   O  = [P~ | Q~] [V ; S]           A from tensor memory, 256 deep
//   KV = W^T K                       A = the weighted V, transposed, from tensor memory
// where Q~_i = 2^{e_i} q_i is exact (a power of two: lam^{i+1} = m_i 2^{e_i}, 1 <= m_i < 2),
// P~_ij = (lam^{i-j} / m_i) P_ij is rounded to bf16 once, and the epilogue multiplies row i
// by so m_i: every term has one rounded factor, P~ or the bf16 copy of S, beside the output's
// own rounding.  A row factor on the state's part alone would cost a second accumulator or
// a round trip of O; a rounded Q~ a second rounding.  When no sequence has more than one chunk
// the second stage is empty: there P~ and S get a second bf16 part each, and only the output's
// rounding is left (the error of a few tokens averages over few values; relative, it is 1.7e-3
// where one part gives 2.4e-3).  In the kernels for all lengths the same rule by sequence costs
// the backward of 4 x 4096 tokens 4 to 10 %, by its registers alone.
//
// The state is held in fp32 registers, and W = w lam^{..} v has fp32 accuracy: the weight is
// split into bf16 numbers w1 + w2 + w3 (8 bits each), and
//   w v = h + l + p + r,   h = bf16(w1 v),  l = w1 v - h,  p = bf16(w2 v),
//                          r = bf16(w3 v + (w2 v - p)),
// where l and w2 v - p are exact in bf16 (a 16-bit product less its upper half).  Each part is
// one or two packed bf16 instructions for two tokens, and KV is four products.  (Two parts
// leave 2^-17, which shows in the fp32 states.)  KV is formed alone for each chunk and added
// in the registers with one rounding: accumulating in tensor memory over a long sequence would
// add up the tensor core's truncations.  lam^L is kept to 48 bits, for the same reason.
//
// No product waits for another chunk's epilogue but through the buffers it needs, so the warps
// run as a pipeline over chunks: 8 warps turn P into P~ and build Q~, 8 build W, 8 hold the
// state, publish its bf16 copy and write O, and four issue the loads, the stores and the three
// products.  Tensor memory holds two P buffers, O and W; KV takes the P buffer that the chunk
// before has finished with.
//
// Shared memory: K and V have two stages; Q has one tile, free again once Q~ is in tensor memory
// (P was formed before), and the output a tile of its own, so that no tile waits for an output to
// leave.  (Q in two stages, its tile taking the output: 109 instead of 105 us for the forward
// below, 396 instead of 352 us for the backward of 4 x 4096 tokens.)  A pair's exchange takes
// some 3000 cycles: the epilogue reads its own half and frees O before it waits for the other
// (backward 352 -> 342 us).  The partial sums cross in fp32, stored straight into the peer's tile:
// in fp16 with a power of two for 32 columns the backward took as long (322 us alone after a flush,
// now 316; among other passes, at the clock that the load leaves, 328 and 337), and columns far below
// the largest, or beside an infinity, were lost.
//
// What bounds it (4 x 4096 tokens, 16 / 32 heads: 106 us among other passes, with the states 3.9 TB/s
// or 0.58 of the measured copy rate): the steps of a chunk that wait on each other.  A chunk takes 5300 cycles, of which the
// tensor pipe works for 3584 (QK 8 products of 64 cycles, O 16, KV 32).  Over two chunks O(c - 1)
// frees the buffer for KV(c), whose end frees it for P(c + 1), from which P~ and then O(c + 1)
// follow; each hand-over crosses tensor memory, and every step shares the SM's one data path with
// the products' operands (256 KB a chunk) and the tiles' arrival.  Without effect: two or three
// parts for W (by truncation or by error-free sums), also with all of a chunk's W ahead of KV;
// finer W buffers; arrivals once a warp; P's factors in registers.  Slower: rows of O written
// straight from registers (126 us), Q's tile freed before P is formed (113 us).
#include <float.h>
#include <stddef.h>
#include <string.h>

#include <initializer_list>

#include "gdn_epi.cuh"
#include "gdn_linear.h"
#include "gdn_tma.h"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kC = 128;                     // tokens of a chunk
constexpr uint32_t kHalf = kC * 128;        // a 128 x 64 bf16 sub-tile
constexpr uint32_t kTile = 2 * kHalf;       // a 128 x 128 tile
constexpr int kGroupP = 8, kGroupW = 8, kGroupS = 8;  // warps of the three groups
constexpr int kWarpLoad = kGroupP + kGroupW + kGroupS;
constexpr int kThreads = (kWarpLoad + 4) * 32;

// Registers a thread: the state's warps hold 64 floats and 32 of an output each, P's a row of Q~.
// The groups' shares must not exceed what the launch gives (kThreads * kRegsLaunch, checked there
// too), or the increase would never end.  (P 80, W 48, state 104: backward of 4 x 4096 tokens 332
// instead of 322 us, by spills of the pairs' epilogue; P 72 or W 32 for more elsewhere: slower.)
constexpr int kRegsLaunch = 72, kRegsP = 80, kRegsW = 40, kRegsState = 112, kRegsIssue = 40;
static_assert(kGroupP * kRegsP + kGroupW * kRegsW + kGroupS * kRegsState + 4 * kRegsIssue <=
                      (kWarpLoad + 4) * kRegsLaunch &&
                  kRegsW <= kRegsP,   // in the state pass P's warps do W's work, with W's share
              "register shares");

// Tensor-memory columns
constexpr uint32_t kColP = 0;      // two buffers of 128: P fp32; then, per half h of 64: P~ of tokens
                                   // 64 h .. in 32 columns and Q~ of features 64 h .. in the next 32
constexpr uint32_t kColX = 256;    // O
constexpr uint32_t kColW = 384;    // two buffers of 64: 32 tokens of W, four parts of 16 (the state
                                   // pass has two more in the second P buffer)
constexpr uint32_t kCols = 512;

struct LinSmem {
    unsigned char k[2][kTile], v[2][kTile];               // TMA tiles, two stages
    unsigned char q[kTile];                               // free again once P is formed and Q~ read
    unsigned char x[kTile];                               // the output on its way (pair mode: the peer's part of
                                                          // this CTA's half, fp32; then the half in plane 1)
    unsigned char s[kTile];                               // bf16 copy of S, row r K-major
    bf16 wtab[3][kC];     // weights of a whole chunk's tokens, three parts
    float ptab[32];       // decays inside a block of 32 columns of P
    float full_hi, full_lo, part_hi, part_lo;  // lam^128 and lam^(partial chunk), head and tail
    uint64_t full_vk[2], v_ok[2], p_done[2], pt_ready[2], w_ready[4], w_free[4], kv_done[2], kv_free[2], o_done[2];
    uint64_t full_q, s_ready, o_free, o_staged, x_free, factors, drain[3];
    // pair mode: the peer may take this CTA's half of the next output; the peer's half is here
    uint64_t peer_ok, rx_full;
    uint32_t tmem_base;
    int dead;
};
static_assert(offsetof(LinSmem, s) % 1024 == 0, "SW128 tiles on 1024-byte boundaries");
static_assert(sizeof(LinSmem) + 1024 <= 232448, "one CTA per SM");

struct LinMaps {
    struct Pass {
        CUtensorMap q, k, v, o;
    } pass[3];
};

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// Descriptor offset (16-byte units) of the x-th 16-deep step of a K-major tile.
__device__ __forceinline__ constexpr uint64_t k_step(int x) { return ((x >> 2) * kHalf + (x & 3) * 32) >> 4; }

// Column of the x-th 16-deep step of P~ (Q~: 32 further on).
__device__ __forceinline__ constexpr uint32_t a_step(int x) { return kColP + 64 * (x >> 2) + 8 * (x & 3); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t x;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
    return x;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t x;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
    return x;
}

// Four 8 x 8 bf16 matrices of shared rows, each transposed: register m of lane l holds
// (row 2 (l % 4) + {0, 1}, column l / 4) of matrix m, whose rows lanes 8 m .. 8 m + 7 point at.
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 8 columns: register 2 k + e of lane t goes to lane t / 4 + 8 e, column 4 k + t % 4.
__device__ __forceinline__ void tmem_st16x128_x2(uint32_t taddr, const uint32_t (&u)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3])
                 : "memory");
}

// ---- the other CTA of a cluster
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Hands over a place whose reads have completed, and nothing that was written: relaxed (a release
// to the cluster takes about a thousand cycles; backward of 4 x 4096 tokens 343 -> 332 us).  The
// memory model does not order those reads before the peer's stores; a dependency does.  Each value
// read is part of a sum that the same lane stores (write32) before it arrives on o_staged, which
// comes before this; a value that is not stored (a row past the sequence) may be anything.
__device__ __forceinline__ void remote_arrive(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_rank(smem_u32(bar), rank))
                 : "memory");
}
// Sixteen bytes into another CTA's shared memory; completes on that CTA's barrier.
__device__ __forceinline__ void remote_store(uint32_t to, const float *x, uint32_t bar) {
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
        "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "r"(bar)
        : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A bounded wait that also gives up once any role of the CTA has.  The timer and the flag
// are looked at every 32 polls only: the timer's reads are slow.
template <bool kCluster = false>
__device__ __forceinline__ bool wait(LinSmem &sm, uint64_t *bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t polls = 1;; ++polls) {
        if (kCluster ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (polls % 32) continue;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (*(volatile int *)&sm.dead || now - t0 > kWaitLimitNs) {
            *(volatile int *)&sm.dead = 1;
            return false;
        }
    }
}

// The same for a whole warp: every lane gets one answer, so that the warp stays together.
__device__ __forceinline__ bool wait_warp(LinSmem &sm, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(sm, bar, parity));
}

__device__ __forceinline__ bool wait_warp_cluster(LinSmem &sm, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait<true>(sm, bar, parity));
}

// What bf16 leaves of 8 values, as bf16 (nothing of an infinity, which the first part holds).
__device__ __forceinline__ uint4 second_part(const float *x) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = x[j] - bf2f(f2bf(x[j]));
        y[j] = y[j] == y[j] ? y[j] : 0.f;
    }
    return make_uint4(epi::pack_bf2(y[0], y[1]), epi::pack_bf2(y[2], y[3]), epi::pack_bf2(y[4], y[5]),
                      epi::pack_bf2(y[6], y[7]));
}

// e^{g n} as head + tail, 48 bits.  The head is rounded towards zero and the tail at least the
// smallest number, so that both keep the sign of an infinite state (y hi + y lo is +-inf, not NaN);
// a power that fp32 has no number for counts as the smallest too, unless e^g itself is zero.
struct Decay {
    float hi, lo;
};
__device__ __forceinline__ Decay decay_power(float g, double n) {
    const float least = expf(g) == 0.f ? 0.f : __int_as_float(1);   // 2^-149
    const double x = exp((double)g * n);
    const float hi = __double2float_rz(x), lo = (float)(x - (double)hi);
    return {hi < least ? least : hi, lo < least ? least : lo};   // (a NaN stays)
}

struct Walk {      // the chunks of this CTA's segment, in scan order
    int t0, len, total;   // the sequence: first token, tokens, chunks
    int first, n;         // the segment: first chunk in scan order, chunks
    __device__ __forceinline__ int chunk(int c, bool rev) const {
        return rev ? total - 1 - (first + c) : first + c;
    }
    __device__ __forceinline__ int start(int c, bool rev) const { return t0 + chunk(c, rev) * kC; }
    __device__ __forceinline__ int length(int c, bool rev) const { return min(kC, len - chunk(c, rev) * kC); }
};

// Columns of chunk c's KV: the P buffer of chunk c - 1, whose readers end with O of that chunk
// and which chunk c + 1 needs next; so KV waits for no epilogue.  The state pass has no outputs
// and takes two regions in turns.
template <int kMode>
__device__ __forceinline__ uint32_t col_kv(int c) {
    return kMode != 2 ? kColP + 128 * ((c + 1) & 1) : c & 1 ? kColP : kColX;
}
__device__ __forceinline__ uint32_t col_w(int b) { return b < 2 ? kColW + 64 * b : kColP + 128 + 64 * (b - 2); }

// lam^{i+1} (forward) or lam^{L-1-i} (reverse) as 2^{e + f}, e whole and 0 <= f < 1.
template <bool kReverse>
__device__ __forceinline__ void read_power(float g2, int i, int L, float &e, float &f) {
    const float x = g2 * (float)(kReverse ? max(L - 1 - i, 0) : i + 1);
    e = floorf(x);
    f = x - e;
}

// 32 columns of output row r: times the row's factor, and out (element `at` of the output, or
// columns 32 h .. of the swizzled bf16 row `place` in shared memory when staged).
__device__ __forceinline__ void scale32(float (&x)[32], float scale) {
    const uint64_t s2 = pair(scale, scale);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 y = unpair(mul2(s2, pair(x[j], x[j + 1])));
        x[j] = y.x;
        x[j + 1] = y.y;
    }
}
__device__ __forceinline__ void write32(const LinearPass &a, const float (&x)[32], size_t at, bool mine,
                                        bool staged, unsigned char *place, int r, int h) {
    if (a.part) {
        if (mine) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(a.part + at + 4 * j) =
                    make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        }
        return;
    }
    uint4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        y[j] = make_uint4(epi::pack_bf2(x[8 * j], x[8 * j + 1]), epi::pack_bf2(x[8 * j + 2], x[8 * j + 3]),
                          epi::pack_bf2(x[8 * j + 4], x[8 * j + 5]), epi::pack_bf2(x[8 * j + 6], x[8 * j + 7]));
    if (staged) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(place + (((4 * h + j) ^ (r & 7)) << 4)) = y[j];
    } else if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(a.o + at + 8 * j) = y[j];
    }
}

// Place of 16 bytes, unit j of row r, of the peer's columns 32 h ..: the 4 KB of one warp's rows
// cover the chunks of plane 1 that write32 stages from that warp, and the same of plane 0.  Four
// rows are 64 bytes side by side (one row's alone: backward of 4 x 4096 tokens 417 us).
__device__ __forceinline__ uint32_t exchange_place(int r, int h, int j) {
    const int at = 8 * (j & 3) + (((r >> 2) & 1) << 2) + ((r & 31) >> 3);
    return (j >> 2) * kHalf + ((r & ~31) + at) * 128 + (((4 * h + (r & 3)) ^ (at & 7)) << 4);
}

// One scan of one (sequence, value head).  kMode 0: outputs and states.  1: outputs summed
// over the two value heads of a cluster of two CTAs.  2: only the states, of every segment but
// a sequence's last (their sums are the start states of the segments that a second launch
// walks at once).  kOne: no sequence has more than one chunk.
template <bool kReverse, int kMode, bool kOne = false>
__device__ __forceinline__ void scan(const LinearArgs &a, const LinearPass &ps, const LinMaps::Pass &maps,
                                     const int hv, const int item) {
    constexpr bool kPair = kMode == 1, kState = kMode == 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    LinSmem &sm = smem_struct<LinSmem>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int n = item, seg = 0, nseg = 1;
    Walk wk;
    if (a.N <= kLinearOrder) {
        int x = 0;
        for (int step = kLinearOrder / 2; step; step >>= 1)   // the last x with seg_first[x] <= item
            if (x + step < a.N && a.seg_first[x + step] <= item) x += step;
        n = a.order[x];
        seg = item - a.seg_first[x];
        nseg = a.seg_first[x + 1] - a.seg_first[x];
        // the host's extents are walked; a device copy that differs is flagged
        wk.t0 = a.cu[n];
        wk.len = a.cu[n + 1] - wk.t0;
        if (tid == kThreads - 1 && (a.cu_dev[n] != wk.t0 || a.cu_dev[n + 1] != wk.t0 + wk.len) && a.status)
            atomicOr(a.status, GDN_DEVICE_CU_SEQLENS_MISMATCH);
    } else {
        // the device's extents, within the buffers; the first CTA compares all of them (below)
        wk.t0 = a.cu_dev[n];
        wk.len = a.cu_dev[n + 1] - wk.t0;
        if (wk.t0 < 0 || wk.len < 0 || wk.t0 > a.T - wk.len || wk.len > a.longest) {
            if (tid == 0 && a.status) atomicOr(a.status, GDN_DEVICE_CU_SEQLENS_MISMATCH);
            return;
        }
    }
    if (kState && seg == nseg - 1) return;
    wk.total = (wk.len + kC - 1) / kC;
    wk.first = seg * a.seg_chunks;
    wk.n = nseg > 1 ? min(a.seg_chunks, wk.total - wk.first) : wk.total;
    if (kOne) wk.n = min(wk.n, 1);   // (as the host has checked)
    const float g = a.log_decay[hv] < -1e4f ? -1e4f : a.log_decay[hv];
    const float g2 = g * 1.4426950408889634f;
    bool cut = false;
    if (kState && g2 * (float)(wk.n * kC) < -150.f) {
        // tokens whose weight at the segment's end is below 2^-150, which is zero in fp32
        const int need = (int)ceilf(-150.f / (g2 * kC));
        cut = need < wk.n;
        if (cut) {
            wk.first += wk.n - need;
            wk.n = need;
        }
    }

    const int hq = hv / (a.HV / ps.nq), hk = hv / (a.HV / ps.nk), hw = hv / (a.HV / ps.nv);
    auto load = [&](const CUtensorMap *map, unsigned char *to, int head, int t, uint64_t *bar) {
        for (int h = 0; h < 2; ++h) tma_load_3d(to + h * kHalf, map, 64 * h, head, t, bar);
    };
    auto load_vk = [&](int c) {
        const int s = c & 1, t = wk.start(c, kReverse);
        mbar_arrive_expect_tx(&sm.full_vk[s], 2 * kTile);
        load(&maps.v, sm.v[s], hw, t, &sm.full_vk[s]);
        load(&maps.k, sm.k[s], hk, t, &sm.full_vk[s]);
        // tiles whose places are still taken start towards L2 (further ahead is slower)
        for (int h = 0; h < 2; ++h) {
            if (c + 2 < wk.n) {
                tma_prefetch_3d(&maps.v, 64 * h, hw, wk.start(c + 2, kReverse));
                tma_prefetch_3d(&maps.k, 64 * h, hk, wk.start(c + 2, kReverse));
            }
            if (!kState) tma_prefetch_3d(&maps.q, 64 * h, hq, t);
        }
    };
    auto load_q = [&](int c) {
        mbar_arrive_expect_tx(&sm.full_q, kTile);
        load(&maps.q, sm.q, hq, wk.start(c, kReverse), &sm.full_q);
    };
    if (warp == kWarpLoad) {
        if (elect_one()) {
            if (wk.n > 0) tma_prefetch_maps(maps);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.full_vk[i], 1);
                mbar_init(&sm.v_ok[i], kGroupW * 32);
                mbar_init(&sm.p_done[i], 1);
                mbar_init(&sm.pt_ready[i], kGroupP * 32);
                mbar_init(&sm.kv_done[i], 1);
                mbar_init(&sm.kv_free[i], kGroupS * 32);
                mbar_init(&sm.o_done[i], 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&sm.w_ready[i], kGroupW * 16);
                mbar_init(&sm.w_free[i], 1);
            }
            mbar_init(&sm.full_q, 1);
            mbar_init(&sm.s_ready, kGroupS * 32);
            mbar_init(&sm.o_free, kGroupS * 32);
            mbar_init(&sm.o_staged, kGroupS * 32);
            mbar_init(&sm.x_free, 1);
            mbar_init(&sm.factors, 1);
            mbar_init(&sm.peer_ok, 1);
            mbar_init(&sm.rx_full, 1);
            for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
            sm.dead = 0;
            fence_mbar_init();
            fence_proxy_async_smem();
            for (int c = 0; c < min(2, wk.n); ++c) {   // before anything else is set up
                load_vk(c);
                if (!kState && c == 0) load_q(c);
            }
        }
        __syncwarp();
    } else if (warp == kWarpLoad + 1) {
        tmem_alloc(&sm.tmem_base, kCols);
        tmem_relinquish();
    }
    if (tid < kC) {
        float w = ps.w * exp2f(g2 * (float)(kReverse ? tid + 1 : kC - 1 - tid));
        for (int x = 0; x < 3; ++x) {
            const bf16 y = f2bf(w);
            sm.wtab[x][tid] = y;
            w -= bf2f(y);
        }
        if (tid < 32) sm.ptab[tid] = exp2f(g2 * (float)(kReverse ? tid : 31 - tid));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (kPair) cluster_sync();   // the peer's barriers are initialised
    const uint32_t tb = sm.tmem_base;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;

    if (!kState && warp < kGroupP) {
        // ---------------------------------------------------------- P~ and Q~
        regs_up<kRegsP>();
        const int quad = warp & 3, half = warp >> 2;   // rows 32 quad .., columns 64 half ..
        const int i = quad * 32 + lane;
        const float at = (float)lane, lw = log2f(ps.w);   // w > 0
        auto second = [&](int j) {   // 8 columns of P~'s second part
            return reinterpret_cast<uint4 *>(sm.k[1] + half * kHalf + sw128_off(i, j));
        };
        for (int c = 0; c < wk.n; ++c) {
            const uint32_t mine = tb + lanes + kColP + 128 * (c & 1) + 64 * half;
            const int L = wk.length(c, kReverse);
            float e, f;
            read_power<kReverse>(g2, i, L, e, f);
            // Q~ first, while P is formed; it waits in registers for its columns
            if (!wait_warp(sm, &sm.full_q, c & 1)) break;
            const unsigned char *qt = sm.q + half * kHalf;
            const __nv_bfloat162 pw = __float2bfloat162_rn(
                e < -120.f ? 0.f : __int_as_float(((int)e + 127) << 23));
            float q[32];
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint4 z = *reinterpret_cast<const uint4 *>(qt + sw128_off(i, 8 * p));
                const uint32_t zz[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&zz[y]), pw);
                    q[4 * p + y] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&t));
                }
            }
            if (!wait_warp(sm, &sm.p_done[c & 1], (c >> 1) & 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int b2 = 0; b2 < 2; ++b2) {   // columns j = 32 b + jj
                const int b = 2 * half + b2;
                float x[16];
                uint32_t *u = reinterpret_cast<uint32_t *>(x);
                if (kReverse ? b < quad : b > quad) {
#pragma unroll
                    for (int p = 0; p < 16; ++p) u[p] = 0u;
                    if (kOne) {
#pragma unroll
                        for (int p = 0; p < 32; p += 8) *second(32 * b2 + p) = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    float r[32];
                    tmem_ld32(mine + 32 * b2, r);
                    tmem_ld_wait();
                    if (b == quad) {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) {
                            const float d = kReverse ? (float)jj - at : at - (float)jj;
                            const float y = r[jj] * ex2(fmaf(g2, d, lw - f));
                            r[jj] = d >= 0.f ? y : 0.f;
                        }
                    } else {
                        const float row = ex2(fmaf(g2, (float)(kReverse ? 32 * b - i : i - 32 * b - 31), lw - f));
                        const uint64_t row2 = pair(row, row);
#pragma unroll
                        for (int jj = 0; jj < 32; jj += 4) {
                            const float4 t = *reinterpret_cast<const float4 *>(&sm.ptab[jj]);
                            const float2 y = unpair(mul2(pair(r[jj], r[jj + 1]), mul2(row2, pair(t.x, t.y))));
                            const float2 z = unpair(mul2(pair(r[jj + 2], r[jj + 3]), mul2(row2, pair(t.z, t.w))));
                            r[jj] = y.x;
                            r[jj + 1] = y.y;
                            r[jj + 2] = z.x;
                            r[jj + 3] = z.y;
                        }
                    }
                    if (kReverse && L < kC) {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) r[jj] = 32 * b + jj < L ? r[jj] : 0.f;
                    }
                    if (kOne) {
#pragma unroll
                        for (int p = 0; p < 32; p += 8) *second(32 * b2 + p) = second_part(r + p);
                    }
#pragma unroll
                    for (int p = 0; p < 16; ++p) u[p] = epi::pack_bf2(r[2 * p], r[2 * p + 1]);
                }
                tmem_st16(mine + 16 * b2, x);   // over columns that this warp has read
            }
            tmem_st32(mine + 32, q);
            if (kOne) fence_proxy_async_smem();
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.pt_ready[c & 1]);
        }
    } else if (warp < kGroupP + kGroupW) {
        // ---------------------------------------------------------- W
        // Half h of the group fills buffer h with the 32-token quarters h and h + 2; in the state
        // pass P's warps take the quarters 2 and 3, with buffers of their own.
        regs_down<kRegsW>();
        const int quad = warp & 3, half = warp < kGroupP ? 2 + (warp >> 2) : (warp - kGroupP) >> 2;
        const uint32_t buf = tb + lanes + col_w(half);
        // this lane's row of the first quarter, and the four 8-feature chunks of the warp in it
        // (rows: 8 tokens of the first or second half of 16; chunks: the first or last 16 features)
        const uint32_t vrow = smem_u32(sm.v[0] + (quad >> 1) * kHalf) +
                              (32 * half + 8 * ((lane >> 3) & 1) + (lane & 7)) * 128;
        uint32_t chunk[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            chunk[x] = (uint32_t)((4 * (quad & 1) + 2 * x + (lane >> 4)) ^ (lane & 7)) * 16;
        bool ok = true;
        for (int c = 0; c < wk.n && ok; ++c) {
            const int s = c & 1, L = wk.length(c, kReverse);
            if (!(ok = wait_warp(sm, &sm.full_vk[s], (c >> 1) & 1))) break;
            if (L < kC) {
                // rows past the sequence hold the next one's tokens: zeros instead (each half
                // clears its own quarters of K, which the product of a quarter waits for)
                for (int x = quad * 32 + lane; x < (kState ? 1 : 2) * 32 * 16; x += kGroupW * 16) {
                    const int y = x >> 4, row = (y >> 5) * 64 + half * 32 + (y & 31), h = (x >> 3) & 1;
                    if (row < L) continue;
                    const uint32_t at = h * kHalf + sw128_off(row, 8 * (x & 7));
                    *reinterpret_cast<uint4 *>(sm.k[s] + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(sm.v[s] + at) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            if (!kState) mbar_arrive(&sm.v_ok[s]);
            // a forward scan's partial chunk ends with the same weights as a whole one
            const int first = 32 * half + 2 * (lane & 3), shift = kReverse ? 0 : kC - L;
            const uint32_t vt = vrow + s * kTile;
#pragma unroll 1
            for (int pass = 0; pass < (kState ? 1 : 2); ++pass) {
                const int use = kState ? c : 2 * c + pass;
                if (use > 0 && !(ok = wait_warp(sm, &sm.w_free[half], (use - 1) & 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int k16 = 0; k16 < 2; ++k16) {   // 16 tokens
                    __nv_bfloat162 w[2][3];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int x = 0; x < 3; ++x)
                        {
                            const int t = first + 64 * pass + 16 * k16 + 8 * k + shift;   // (past the sequence: any)
                            if (shift & 1)
                                w[k][x] = __nv_bfloat162(sm.wtab[x][min(t, kC - 1)], sm.wtab[x][min(t + 1, kC - 1)]);
                            else
                                w[k][x] = *reinterpret_cast<const __nv_bfloat162 *>(&sm.wtab[x][min(t, kC - 2)]);
                        }
                    uint32_t in[2][4];
                    ldmatrix4t(vt + (64 * pass + 16 * k16) * 128 + chunk[0], in[0]);
                    ldmatrix4t(vt + (64 * pass + 16 * k16) * 128 + chunk[1], in[1]);
                    if (L < kC) {   // tokens past the sequence
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int left = L - (64 * pass + 32 * half + 16 * k16 + 8 * k + 2 * (lane & 3));
                            const uint32_t keep = left > 1 ? 0xffffffffu : left > 0 ? 0xffffu : 0u;
#pragma unroll
                            for (int x = 0; x < 4; ++x) in[x >> 1][k + 2 * (x & 1)] &= keep;
                        }
                    }
#pragma unroll
                    for (int g16 = 0; g16 < 2; ++g16) {   // features 32 quad + 16 g16 ..
                        uint32_t part[4][4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {   // 8 tokens x & 1, features 8 (x >> 1) ..
                            const __nv_bfloat162 *wx = w[x & 1];
                            const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162 *>(&in[g16][x]);
                            const __nv_bfloat162 h = __hmul2(wx[0], v2);
                            const __nv_bfloat162 l = __hfma2(wx[0], v2, __hneg2(h));
                            const __nv_bfloat162 p = __hmul2(wx[1], v2);
                            const __nv_bfloat162 r = __hfma2(wx[2], v2, __hfma2(wx[1], v2, __hneg2(p)));
                            const int at = 2 * (x & 1) + (x >> 1);
                            part[0][at] = *reinterpret_cast<const uint32_t *>(&h);
                            part[1][at] = *reinterpret_cast<const uint32_t *>(&l);
                            part[2][at] = *reinterpret_cast<const uint32_t *>(&p);
                            part[3][at] = *reinterpret_cast<const uint32_t *>(&r);
                        }
                        const uint32_t at = buf + ((uint32_t)(16 * g16) << 16) + 8 * k16;
#pragma unroll
                        for (int y = 0; y < 4; ++y) tmem_st16x128_x2(at + 16 * y, part[y]);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sm.w_ready[half]);
            }
        }
    } else if (warp < kWarpLoad) {
        // ---------------------------------------------------------- state and output
        regs_up<kRegsState>();
        const int x0 = warp - kGroupP - kGroupW;
        const int r = (warp & 3) * 32 + lane, col = (x0 >> 2) * 64;  // row of S and of O; columns
        // state x of `of`, or none where the checked build finds it outside
        auto state_of = [&](float *base, long long x, long long of) {
            const bool in = base && in_range((x * a.HV + hv) * kDim * kDim, kDim * kDim, of * a.HV * kDim * kDim, a.status);
            return in ? base + ((size_t)x * a.HV + hv) * kDim * kDim : nullptr;
        };
        const float *src = state_of(const_cast<float *>(ps.s0), n, a.N);
        float *dst = state_of(ps.s1, n, a.N);
        if (a.pool) {
            const int slot = a.pool_idx[n];
            if (slot >= a.num_slots && r == 0 && a.pool_status) *a.pool_status = 1;
            if (slot > 0 && slot < a.num_slots) {
                dst = state_of(a.pool, slot, a.num_slots);
                src = (!a.pool_resume || a.pool_resume[n]) ? dst : nullptr;
            }
        }
        float *keep_start = nullptr;
        bool src_rows = ps.rows, dst_rows = ps.rows;   // row r contiguous, or column c
        if (nseg > 1) {   // inner states of a split sequence: after segment k in record `first + k`
            if (seg > 0) {
                src = kState ? nullptr : state_of(ps.seg_state, item - 1, a.items);
                src_rows = ps.seg_rows;
            }
            // a pool slot is written by its last segment's CTA, perhaps before the first one's
            // starts: the state pass keeps the start state in the last record, which is free
            float *kept = seg == 0 && a.pool ? state_of(ps.seg_state, item + nseg - 1, a.items) : nullptr;
            if (seg == 0 && a.pool && !kState) {
                src = kept;
                src_rows = ps.seg_rows;
            }
            keep_start = kState ? kept : nullptr;
            if (kState) {
                dst = state_of(ps.seg_state, item, a.items);
                dst_rows = ps.seg_rows;
            } else if (seg < nseg - 1) {
                dst = nullptr;
            }
        }
        float st[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) st[j] = 0.f;
        if (src) {
            if (src_rows) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float4 z = *reinterpret_cast<const float4 *>(src + (size_t)r * kDim + col + 4 * j);
                    st[4 * j] = z.x;
                    st[4 * j + 1] = z.y;
                    st[4 * j + 2] = z.z;
                    st[4 * j + 3] = z.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) st[j] = src[(size_t)(col + j) * kDim + r];
            }
        }
        if (keep_start) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                *reinterpret_cast<float4 *>(keep_start + (size_t)r * kDim + col + 4 * j) =
                    make_float4(st[4 * j], st[4 * j + 1], st[4 * j + 2], st[4 * j + 3]);
        }
        if (cut) {   // the start state too, but for infinities and NaN
            const float one = expf(g);
#pragma unroll
            for (int j = 0; j < 64; ++j) st[j] = fabsf(st[j]) <= FLT_MAX ? 0.f : one * st[j];
        }
        unsigned char *srow = sm.s + (col >> 6) * kHalf;
        auto publish = [&]() {
            epi::put_row32(srow, r, 0, st);
            epi::put_row32(srow, r, 32, st + 32);
            fence_proxy_async_smem();
            mbar_arrive(&sm.s_ready);
        };
        if (kOne) {
#pragma unroll
            for (int j = 0; j < 64; j += 8)
                *reinterpret_cast<uint4 *>(sm.v[1] + (col >> 6) * kHalf + sw128_off(r, j)) = second_part(st + j);
        }
        if (!kState && wk.n > 0) publish();
        auto store_state = [&]() {
            if (!dst) return;
            if (dst_rows) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<float4 *>(dst + (size_t)r * kDim + col + 4 * j) =
                        make_float4(st[4 * j], st[4 * j + 1], st[4 * j + 2], st[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) dst[(size_t)(col + j) * kDim + r] = st[j];
            }
        };
        const bool have = wk.n == 0 || wait_warp(sm, &sm.factors, 0);
        for (int c = 0; have && c < wk.n; ++c) {
            const int s = c & 1, L = wk.length(c, kReverse);
            const float fh = L < kC ? sm.part_hi : sm.full_hi, fl = L < kC ? sm.part_lo : sm.full_lo;
            if (!wait_warp(sm, &sm.kv_done[s], (c >> 1) & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[32];
                tmem_ld32(tb + lanes + col_kv<kMode>(c) + col + 32 * h, x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const uint64_t y = pair(st[32 * h + j], st[32 * h + j + 1]);
                    const float2 z = unpair(fma2(y, pair(fh, fh), fma2(y, pair(fl, fl), pair(x[j], x[j + 1]))));
                    st[32 * h + j] = z.x;
                    st[32 * h + j + 1] = z.y;
                }
            }
            tc_fence_before();
            mbar_arrive(&sm.kv_free[s]);
            if (c + 1 == wk.n) store_state();   // while the last O runs
            if (kState) continue;
            if (!wait_warp(sm, &sm.o_done[s], (c >> 1) & 1)) break;
            tc_fence_after();
            float e, f;
            read_power<kReverse>(g2, r, L, e, f);
            const float scale = ps.so * ex2(f);
            const uint32_t from = tb + lanes + kColX + col;
            const int first = kPair ? 64 * (hv & 1) + (col >> 1) : col;   // this warp's first column to write
            const size_t out = (((size_t)wk.start(c, kReverse) + r) * ps.no + (kPair ? hv >> 1 : hv)) * kDim + first;
            const bool staged = L == kC && !ps.part;   // whole chunks of bf16 leave by TMA
            const bool mine = r < L && in_range(out, kPair ? 32 : 64, (long long)a.T * ps.no * kDim, a.status);
            unsigned char *orow = sm.x + (kPair ? kHalf : (col >> 6) * kHalf) + r * 128;
            if (kPair) {
                // Each CTA writes 64 columns of the pair's sum; the other 64 go to the peer.
                if ((col >> 6) != (hv & 1)) {
                    if (!wait_warp_cluster(sm, &sm.peer_ok, c & 1)) break;   // its tile is free
                    const uint32_t peer = (hv & 1) ^ 1;
                    const uint32_t x_peer = map_rank(smem_u32(sm.x), peer), full = map_rank(smem_u32(&sm.rx_full), peer);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x[32];
                        tmem_ld32(from + 32 * h, x);
                        tmem_ld_wait();
                        scale32(x, scale);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            remote_store(x_peer + exchange_place(r, h, j), x + 4 * j, full);
                    }
                }
                if (c + 1 < wk.n) publish();   // while the peer's half comes
                const int h = col >> 6;
                float x[32];
                tmem_ld32(tb + lanes + kColX + first, x);
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive(&sm.o_free);
                if (!wait_warp_cluster(sm, &sm.rx_full, c & 1)) break;
                scale32(x, scale);
#pragma unroll
                for (int j = 0; j < 8; ++j) {   // (two terms: the same sum whichever CTA adds)
                    const float4 y = *reinterpret_cast<const float4 *>(sm.x + exchange_place(r, h, j));
                    x[4 * j] += y.x;
                    x[4 * j + 1] += y.y;
                    x[4 * j + 2] += y.z;
                    x[4 * j + 3] += y.w;
                }
                __syncwarp();
                write32(ps, x, out, mine, staged, orow, r, h);   // (over what its warp has read)
            } else {
                if (c > 0 && !wait_warp(sm, &sm.x_free, (c - 1) & 1)) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[32];
                    tmem_ld32(from + 32 * h, x);
                    tmem_ld_wait();
                    if (h == 1) {
                        tc_fence_before();
                        mbar_arrive(&sm.o_free);
                    }
                    scale32(x, scale);
                    write32(ps, x, out + 32 * h, mine, staged, orow, r, h);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.o_staged);
            if (!kPair && c + 1 < wk.n) publish();
        }
        if (wk.n == 0) store_state();
    } else {
        // ---------------------------------------------------------- issuing warps
        // The whole warp waits and one elected lane issues: the operands stay in uniform
        // registers (issued from a lane's own branch, each product took 80 to 130 cycles
        // to issue, more than the 64 it runs).
        regs_down<kRegsIssue>();
        const int role = __shfl_sync(0xffffffffu, warp, 0) - kWarpLoad;
        if (role == 0) {
            // ------------------------------------------------------ loads
            // pair mode: the exchange tile may take the peer's part of chunk c's output
            auto arm = [&](int c) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sm.rx_full, kTile);
                    remote_arrive(&sm.peer_ok, (hv & 1) ^ 1);
                }
                __syncwarp();
            };
            int issued = min(2, wk.n), armed = min(1, wk.n);
            if (kPair && armed) arm(0);
            for (int c = 0; c < wk.n; ++c) {
                const int s = c & 1, mark = (c >> 1) & 1;
                if (c + 2 < wk.n) {
                    if ((!kState && !wait_warp(sm, &sm.o_done[s], mark)) || !wait_warp(sm, &sm.kv_done[s], mark)) break;
                    if (elect_one()) load_vk(c + 2);
                    __syncwarp();
                    issued = c + 3;
                }
                if (kState) continue;
                if (!wait_warp(sm, &sm.o_staged, c & 1)) break;
                if (elect_one()) {   // (a partial chunk's output has been written)
                    if (wk.length(c, kReverse) == kC && !ps.part) {
                        for (int h = kPair ? 1 : 0; h < 2; ++h)
                            tma_store_3d(&maps.o, kPair ? 64 * (hv & 1) : 64 * h, kPair ? hv >> 1 : hv,
                                         wk.start(c, kReverse), sm.x + h * kHalf);
                        tma_store_commit();
                        tma_store_wait_read();
                    }
                    mbar_arrive(&sm.x_free);
                }
                __syncwarp();
                if (kPair && c + 1 < wk.n) {
                    arm(c + 1);
                    armed = c + 2;
                }
            }
            if (elect_one()) tma_store_wait_all();
            __syncwarp();
            // copies still in flight write this CTA's shared memory: wait for them (bounded)
            for (int c = max(0, issued - 2); c < issued; ++c)
                mbar_wait(&sm.full_vk[c & 1], (c >> 1) & 1, kDrainLimitNs);
            if (kPair && armed) mbar_wait(&sm.rx_full, (armed - 1) & 1, kDrainLimitNs);
        } else if (role == 1) {
            // ------------------------------------------------------ P = Q K^T
            const uint32_t id = idesc_bf16(128, 128, 0, 0);
            const uint64_t qd = sdesc(smem_u32(sm.q), 16, 1024), kd0 = sdesc(smem_u32(sm.k), 16, 1024);
            int issued = kState ? 0 : min(1, wk.n);
            for (int c = 0; !kState && c < wk.n; ++c) {
                const int s = c & 1;
                if (!wait_warp(sm, &sm.full_vk[s], (c >> 1) & 1) || !wait_warp(sm, &sm.full_q, c & 1)) break;
                // (KV of chunk c - 1 took this P buffer after O of chunk c - 2)
                if (c > 0 && !wait_warp(sm, &sm.kv_free[s ^ 1], ((c - 1) >> 1) & 1)) break;
                tc_fence_after();
                const uint64_t kd = kd0 + ((s * kTile) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mma_bf16(tb + kColP + 128 * s, qd + k_step(x), kd + k_step(x), id, x > 0);
                    mma_commit(&sm.p_done[s]);
                }
                __syncwarp();
                // The next Q, once this one is in P and Q~.  (P's warps arrive after Q~ is stored, which
                // took the tile's data: an arrival right after the reads was seen to come before them.)
                if (c + 1 < wk.n) {
                    if (!wait_warp(sm, &sm.pt_ready[s], (c >> 1) & 1)) break;
                    if (elect_one()) load_q(c + 1);
                    __syncwarp();
                    issued = c + 2;
                }
            }
            if (issued > 0) mbar_wait(&sm.full_q, (issued - 1) & 1, kDrainLimitNs);
        } else if (role == 2) {
            // ------------------------------------------------------ O = [P~ | Q~] [V ; S]
            const uint32_t idv = idesc_bf16(128, 128, 0, 1), ids = idesc_bf16(128, 128, 0, 0);
            const uint64_t vd0 = sdesc(smem_u32(sm.v), kHalf, 1024), sd0 = sdesc(smem_u32(sm.s), 16, 1024);
            for (int c = 0; !kState && c < wk.n; ++c) {
                const int s = c & 1;
                if (!wait_warp(sm, &sm.v_ok[s], (c >> 1) & 1) || !wait_warp(sm, &sm.s_ready, c & 1) ||
                    !wait_warp(sm, &sm.pt_ready[s], (c >> 1) & 1) ||
                    (c > 0 && !wait_warp(sm, &sm.o_free, (c - 1) & 1)))
                    break;
                tc_fence_after();
                const uint64_t vd = vd0 + ((s * kTile) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mma_ts(tb + kColX, tb + 128 * s + a_step(x) + 32, sd0 + k_step(x), ids, x > 0);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mma_ts(tb + kColX, tb + 128 * s + a_step(x), vd + 128 * x, idv, true);
                    if (kOne) {   // second parts: S in the second stage's V tile, P~ in its K tile
                        const uint64_t p2 = sdesc(smem_u32(sm.k[1]), 16, 1024), s2 = sdesc(smem_u32(sm.v[1]), 16, 1024);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            mma_ts(tb + kColX, tb + a_step(x) + 32, s2 + k_step(x), ids, true);
                            mma_bf16(tb + kColX, p2 + k_step(x), vd + 128 * x, idv, true);
                        }
                    }
                    mma_commit(&sm.o_done[s]);
                }
                __syncwarp();
            }
        } else {
            // ------------------------------------------------------ KV = W^T K
            const uint32_t id = idesc_bf16(128, 128, 0, 1);
            const uint64_t kd0 = sdesc(smem_u32(sm.k), kHalf, 1024);
            // lam^128 and lam^(partial chunk) to 48 bits, for the state
            if (lane < 2) {
                const Decay x = decay_power(g, lane == 0 ? kC : wk.len % kC);
                (lane == 0 ? sm.full_hi : sm.part_hi) = x.hi;
                (lane == 0 ? sm.full_lo : sm.part_lo) = x.lo;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.factors);
            __syncwarp();
            bool ok = true;
            for (int c = 0; c < wk.n && ok; ++c) {
                const int s = c & 1;
                if (kState ? c > 1 && !wait_warp(sm, &sm.kv_free[s], ((c >> 1) - 1) & 1)
                           : c > 0 && !wait_warp(sm, &sm.o_done[s ^ 1], ((c - 1) >> 1) & 1))
                    break;
                if (!wait_warp(sm, &sm.full_vk[s], (c >> 1) & 1)) break;
                const uint64_t kd = kd0 + ((s * kTile) >> 4);
#pragma unroll
                for (int qd = 0; qd < 4; ++qd) {
                    const int b = kState ? qd : qd & 1, use = kState ? c : 2 * c + (qd >> 1);
                    ok = ok && wait_warp(sm, &sm.w_ready[b], use & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int part = 0; part < 4; ++part)
                                mma_ts(tb + col_kv<kMode>(c), tb + col_w(b) + 16 * part + 8 * x,
                                       kd + 128 * (2 * qd + x), id, qd > 0 || x > 0 || part > 0);
                        mma_commit(&sm.w_free[b]);
                        if (qd == 3) mma_commit(&sm.kv_done[s]);
                    }
                    __syncwarp();
                }
            }
            if (!kState && a.N > kLinearOrder && blockIdx.x == 0 && a.status) {
                uint64_t sum = 0;
                for (int i = lane; i <= a.N; i += 32) sum += offset_term(i, a.cu_dev[i]);
                for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (lane == 0 && sum != a.cu_sum) atomicOr(a.status, GDN_DEVICE_CU_SEQLENS_MISMATCH);
            }
        }
        if (role > 0 && *(volatile int *)&sm.dead) {
            // products in flight read tiles and tensor memory: wait for them (bounded)
            if (elect_one()) mma_commit(&sm.drain[role - 1]);
            __syncwarp();
            mbar_wait(&sm.drain[role - 1], 0, kDrainLimitNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();   // neither CTA leaves while the other may still write to it
    if (tid == 0 && sm.dead && a.status) atomicOr(a.status, GDN_DEVICE_WAIT_TIMEOUT);
    if (warp == kWarpLoad + 1) tmem_dealloc(tb, kCols);
}

// The scans of a call, work items longest first, the passes of an item and its value heads
// side by side (the two CTAs of a cluster are two value heads of one pass).
//   kSet 0: a forward.  1: the state pass.  2, 3: a backward without and with pairs.
template <int kSet, bool kOne>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ LinearArgs a, const __grid_constant__ LinMaps maps) {
    const int hv = blockIdx.x % a.HV, rest = blockIdx.x / a.HV;
    int item, p;
    if (kSet >= 2 && rest >= 2 * a.items) {   // dv's scans, the shortest, fill in at the end
        item = rest - 2 * a.items;
        p = 2;
    } else {
        const int sides = kSet == 0 ? 1 : kSet == 1 ? a.state_passes : 2;
        item = rest / sides;
        p = rest % sides * (kSet == 1 ? 2 : 1);   // (the state pass takes scans 0 and 2)
    }
    if (kSet == 0) {
        scan<false, 0, kOne>(a, a.pass[0], maps.pass[0], hv, item);
    } else if (kSet == 1) {
        if (p) scan<true, 2>(a, a.pass[2], maps.pass[2], hv, item);
        else scan<false, 2>(a, a.pass[0], maps.pass[0], hv, item);
    } else if (kSet == 2) {
        if (p) scan<true, 0, kOne>(a, a.pass[p], maps.pass[p], hv, item);
        else scan<false, 0, kOne>(a, a.pass[0], maps.pass[0], hv, item);
    } else {
        if (p == 0) scan<false, 1, kOne>(a, a.pass[0], maps.pass[0], hv, item);
        else if (p == 1) scan<true, 1, kOne>(a, a.pass[1], maps.pass[1], hv, item);
        else scan<true, 0, kOne>(a, a.pass[2], maps.pass[2], hv, item);
    }
}

// Start states of a split sequence's segments: record k (the state after segment k alone,
// segment 0's from its true start) becomes the state after segments 0 .. k.
__global__ void __launch_bounds__(256) k_linear_stitch(const __grid_constant__ LinearArgs a) {
    const int x = blockIdx.z / a.state_passes, hv = blockIdx.y;
    const int first = a.seg_first[x], nseg = a.seg_first[x + 1] - first;
    if (nseg < 3) return;
    const float g = a.log_decay[hv] < -1e4f ? -1e4f : a.log_decay[hv];
    const Decay lam = decay_power(g, (double)a.seg_chunks * kC);
    const float fh = lam.hi, fl = lam.lo;
    const size_t step4 = (size_t)a.HV * kDim * kDim / 4;
    float *rec = a.pass[blockIdx.z % a.state_passes * 2].seg_state;
    if (!in_range(((long long)first * a.HV + hv) * kDim * kDim, ((long long)(nseg - 2) * a.HV + 1) * kDim * kDim,
                  (long long)a.items * a.HV * kDim * kDim, a.status))
        return;
    float4 *p = reinterpret_cast<float4 *>(rec + ((size_t)first * a.HV + hv) * kDim * kDim) +
                blockIdx.x * 256 + threadIdx.x;
    float4 y = *p;
    for (int k = 1; k < nseg - 1; k += 8) {   // eight records on their way at once
        float4 z[8];
        const int m = min(8, nseg - 1 - k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < m) z[j] = p[(size_t)(k + j) * step4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < m) {
                y.x = fmaf(y.x, fh, fmaf(y.x, fl, z[j].x));
                y.y = fmaf(y.y, fh, fmaf(y.y, fl, z[j].y));
                y.z = fmaf(y.z, fh, fmaf(y.z, fl, z[j].z));
                y.w = fmaf(y.w, fh, fmaf(y.w, fl, z[j].w));
                p[(size_t)(k + j) * step4] = y;
            }
    }
}

using Kernel = void (*)(LinearArgs, LinMaps);

cudaError_t launch_set(Kernel kernel, int scans, bool pairs, const LinearArgs &a, const LinMaps &m, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.items * a.HV * scans);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(LinSmem) + 1024;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = pairs ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, m);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearArgs &a, cudaStream_t s) {
    const bool one = a.longest <= kC, pairs = a.passes > 1 && a.pass[0].pair;
    const Kernel kernel = a.passes == 1 ? (one ? k_linear_tc<0, true> : k_linear_tc<0, false>)
                          : pairs       ? (one ? k_linear_tc<3, true> : k_linear_tc<3, false>)
                                        : (one ? k_linear_tc<2, true> : k_linear_tc<2, false>);
    const Kernel states = k_linear_tc<1, false>;
    const int smem = (int)sizeof(LinSmem) + 1024;
    cudaError_t e;
    for (Kernel k : {kernel, a.seg_chunks > 0 ? states : kernel}) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;   // the groups' register shares rely on it
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        if (a.seg_chunks == 0) break;
    }
    // (the calls above have made the device's context current, which the map encoder needs)
    LinMaps m;
    memset(&m, 0, sizeof(m));
    // a backward's three scans read the same four tensors: each is encoded once
    const bf16 *known[4];
    int known_heads[4];
    const CUtensorMap *map[4];
    int count = 0;
    bool ok = true;
    auto encode = [&](CUtensorMap &x, const bf16 *base, int heads) {
        const uint64_t rowb = kDim * sizeof(bf16);
        ok = ok && encode_rows_bf16(&x, base, heads, a.T, rowb, rowb * heads, kC);
    };
    auto input = [&](CUtensorMap &x, const bf16 *base, int heads) {
        for (int i = 0; i < count; ++i)
            if (known[i] == base && known_heads[i] == heads) {
                x = *map[i];
                return;
            }
        encode(x, base, heads);
        if (count < 4) {
            known[count] = base;
            known_heads[count] = heads;
            map[count++] = &x;
        }
    };
    for (int i = 0; i < a.passes && a.T > 0; ++i) {
        const LinearPass &p = a.pass[i];
        LinMaps::Pass &x = m.pass[i];
        input(x.q, p.q, p.nq);
        input(x.k, p.k, p.nk);
        input(x.v, p.v, p.nv);
        if (p.part) x.o = x.v;   // not used, but fetched with the others
        else encode(x.o, p.o, p.no);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (a.seg_chunks > 0) {
        if ((e = launch_set(states, a.state_passes, false, a, m, s)) != cudaSuccess) return e;
        k_linear_stitch<<<dim3(kDim * kDim / 1024, a.HV, a.N * a.state_passes), 256, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return launch_set(kernel, a.passes, pairs, a, m, s);
}

}  // namespace gdn
