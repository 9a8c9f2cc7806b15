// gdn_rope.cu -- rotary positions of packed heads: half and interleaved layouts, the first
// `rot` elements of each head, forward and gradient.
//
// Pair p of a head at position pos turns by a = 2 pi pos f_p:
//   x1' = m (x1 cos a - x2 sin a),  x2' = m (x2 cos a + x1 sin a),
// and the gradient is the same with -a.  f_p comes in turns per position as the sum of two
// fp32 numbers, so that the fraction of pos f_p keeps about 2^-21 turns at any int32
// position: pos is split into two parts that fp32 holds exactly, each part's product loses
// its whole turns inside one fused multiply-add (rounded once), and only a fraction of a
// turn reaches sincospif.  An fp32 angle would be off by 2^-24 pos radians instead.
//
// Bound by HBM: every element is read and written once, the cosines and sines of a token are formed
// once for all of its heads.  Among other passes, 32768 tokens of 16 + 16 heads take 84 us, 6.4 TB/s
// or 0.94 of the measured copy rate; the gradient of 16384 tokens of 32 + 4 heads of 256, 94 us, 0.95
// of it.  256 tokens take 3 us on the GPU, which the launch hides.
#include <algorithm>

#include "gdn_linear.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float turn_fraction(int32_t pos, float head, float tail) {
    const float lo = (float)(pos & 0xffff), hi = (float)(pos & ~0xffff);  // both exact
    float x = __fmaf_rn(lo, head, -rintf(lo * head));
    x += __fmaf_rn(hi, head, -rintf(hi * head));
    x -= rintf(x);
    x = __fmaf_rn(lo, tail, x);
    x = __fmaf_rn(hi, tail, x);
    return x - rintf(x);
}

// V elements of bf16, loaded and stored at once.
template <int V>
struct alignas(2 * V) Pack {
    bf16 x[V];
};

// One block per `tokens` consecutive tokens: their cosines and sines go to shared memory
// once, for every head.  A unit is V pairs of a head (2V elements): unit j of a head holds
// pairs [jV, jV + V) when jV < rot / 2, else 2V elements past `rot`, which are copied.
template <int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) k_rope(const RopeArgs a, int tokens) {
    extern __shared__ float2 cs[];  // [tokens][rot / 2]
    const int half = a.rot / 2;
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        float s, c;
        sincospif(2.f * turn_fraction(a.pos[t0 + t], a.freq[p], a.freq[half + p]), &s, &c);
        cs[i] = make_float2(a.mscale * c, a.backward ? -a.mscale * s : a.mscale * s);
    }
    __syncthreads();
    using P = Pack<V>;
    const int per_head = a.D / (2 * V), heads = a.Hq + a.Hk, units = heads * per_head;
    for (int i = threadIdx.x; i < nt * units; i += kThreads) {
        const int t = i / units, u = i - t * units;
        const int h = u / per_head, j = u - h * per_head;
        const bool is_q = h < a.Hq;
        const size_t row = is_q ? ((size_t)(t0 + t) * a.Hq + h) * a.D
                                : ((size_t)(t0 + t) * a.Hk + (h - a.Hq)) * a.D;
        if (!in_range(row, a.D, (long long)a.T * (is_q ? a.Hq : a.Hk) * a.D, nullptr)) continue;
        const bf16 *src = (is_q ? a.q : a.k) + row;
        bf16 *dst = (is_q ? a.qo : a.ko) + row;
        const bool turned = j * V < half;
        const int first = turned && !kInterleaved ? j * V : j * 2 * V;
        const int second = turned && !kInterleaved ? half + j * V : first + V;
        P x = *reinterpret_cast<const P *>(src + first), y = *reinterpret_cast<const P *>(src + second);
        if (turned) {
            const float2 *e = cs + t * half + j * V;
            if (kInterleaved) {
                bf16 z[2 * V];
#pragma unroll
                for (int p = 0; p < V; ++p) {
                    z[p] = x.x[p];
                    z[V + p] = y.x[p];
                }
#pragma unroll
                for (int p = 0; p < V; ++p) {
                    const float x1 = bf2f(z[2 * p]), x2 = bf2f(z[2 * p + 1]);
                    z[2 * p] = f2bf(x1 * e[p].x - x2 * e[p].y);
                    z[2 * p + 1] = f2bf(x2 * e[p].x + x1 * e[p].y);
                }
#pragma unroll
                for (int p = 0; p < V; ++p) {
                    x.x[p] = z[p];
                    y.x[p] = z[V + p];
                }
            } else {
#pragma unroll
                for (int p = 0; p < V; ++p) {
                    const float x1 = bf2f(x.x[p]), x2 = bf2f(y.x[p]);
                    x.x[p] = f2bf(x1 * e[p].x - x2 * e[p].y);
                    y.x[p] = f2bf(x2 * e[p].x + x1 * e[p].y);
                }
            }
        }
        *reinterpret_cast<P *>(dst + first) = x;
        *reinterpret_cast<P *>(dst + second) = y;
    }
}

template <int V>
cudaError_t launch_width(const RopeArgs &a, cudaStream_t s) {
    // Up to four tokens a block, for about four units a thread, once every SM has blocks for its
    // eight places all the same (one call alone, by events, its launch included: 32768 tokens of 32
    // heads of 128, 97 us with one, 87 with four; 16384 tokens of 36 heads of 256, nine units a thread
    // with four, 97 and 101).  A decoding step keeps one, to spread over the SMs (256 tokens: 9 us, 11
    // with four).
    const int units = (a.Hq + a.Hk) * (a.D / (2 * V)), places = 8 * 152;
    const int tokens = std::max(1, std::min({4, 4 * kThreads / units, a.T / places}));
    const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);
    const unsigned grid = ((unsigned)a.T + tokens - 1) / tokens;   // (T < 2^31)
    if (a.interleaved) k_rope<V, true><<<grid, kThreads, smem, s>>>(a, tokens);
    else k_rope<V, false><<<grid, kThreads, smem, s>>>(a, tokens);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    // the widest unit whose halves, tail and row are whole units
    auto fits = [&](int v) { return (a.rot / 2) % v == 0 && (a.D - a.rot) % (2 * v) == 0; };
    if (fits(8)) return launch_width<8>(a, s);
    if (fits(4)) return launch_width<4>(a, s);
    if (fits(2)) return launch_width<2>(a, s);
    return launch_width<1>(a, s);
}

}  // namespace gdn
