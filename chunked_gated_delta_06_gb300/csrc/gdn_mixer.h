// gdn_mixer.h -- internal interface of the kernels around a recurrence: the short causal
// convolution, the selective state space scan, the norms with their gate and residual.
#pragma once

#include "gdn_kernels.h"
#include "gdn_linear.h"

namespace gdn {

// The sequences of a packed call.  The kernels read the device's offsets and clamp what they read
// to [0, T], so that no offsets lead them out of a buffer; where the caller has a status word,
// their sum (offset_term) is held against the host's.
struct PackArgs {
    int N, T;
    const int *cu;       // [N + 1] on the device
    uint64_t cu_sum;     // of the host's offsets
    int *status;         // or null
};

// Slots of a pool that hold the states of sequences (rows of a step).
struct SlotArgs {
    int num_slots;
    const int *idx;      // [N] on the device, or null: no pool
    const int *resume;   // [N] or null
    int *status;         // or null: set to 1 when an index >= num_slots was skipped
};

struct ConvArgs {
    PackArgs pack;
    SlotArgs slots;
    int C, W, silu, f32;
    const void *x;            // [T, C], rows x_stride apart
    long long x_stride;
    const float *w, *bias;    // [C, W], [C] or null
    const void *s0;           // [N, C, W - 1] (or the pool's slots), or null
    void *s1;                 // the same, or null
    void *y;                  // [T, C]
    // backward
    const void *dy, *ds1;     // [T, C], [N, C, W - 1] or null
    void *dx, *ds0;           // [T, C], [N, C, W - 1] or null
    float *dw, *dbias;        // [C, W], [C] or null
    float *part;              // [tiles, C, W + 1] sums of a tile's tokens
    int tile, tiles;          // tokens of a tile, tiles of the pack
};
// the backward's tiles (they set the size of its workspace)
inline int conv_bwd_tile() { return 128; }

cudaError_t launch_conv_fwd(ConvArgs a, cudaStream_t s);
cudaError_t launch_conv_bwd(ConvArgs a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs &a, int batch, cudaStream_t s);

// out[i] = sum over r < rows of part[r][i], in an order fixed by the sizes.  Column i goes to
// main[i / per * keep + i % per] where i % per < keep, else to rest, whose runs are the per - keep
// others (null: dropped).
struct FoldArgs {
    const float *part;
    long long rows, cols;
    int per, keep;
    float *main, *rest;
};
cudaError_t launch_fold(const FoldArgs &a, cudaStream_t s);

struct ScanArgs {
    PackArgs pack;
    SlotArgs slots;
    int C, G, Ns, f32;
    const void *x, *dt, *z, *B, *Cm;              // [T, C] and [T, G, Ns]; z or null
    long long xs, dts, zs, bs, cs;                // their elements from token to token
    const float *A_log, *D, *dt_bias;             // [C, Ns], [C] or null
    const float *s0;                              // [N, C, Ns] (or the pool's slots), or null
    float *s1;                                    // the same, or null
    void *y;                                      // [T, C]
    // split scans: records of a segment, by item (see scan_items)
    int seg;                                      // tokens of a segment; > T: not split
    float *rec_h, *rec_d;                         // [items, C, Ns] end states, [items, C] sums of d
    // backward
    const void *dy;
    const float *ds1;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA_log, *dD, *ddt_bias, *ds0;
    float *rec_g;                                 // [items, C, Ns] gradients at the segments' starts
    float *marks, *mark_d;                        // [marks, C, Ns] states ahead of each tile; [marks, C], if split
    float *part_bc;                               // [blocks of a group, T, G, 2 Ns]
    float *part_c;                                // [items, C, Ns + 2]: dA, dD, ddt_bias
};
// Work items of a scan: sequence n has those from n + cu[n] / seg on, one more than its whole
// segments fit at most; those past its end are idle.
inline long long scan_items(int N, long long T, int seg) { return N + T / seg; }

// Rows of a block of the steps, which walk their rows one after another: those that end soonest, in waves of
// the blocks that run at once (a wave takes about a row's time before its first one).
inline int step_rows(int batch, int across, int at_once) {
    int best = 1;
    long long least = 1LL << 62;
    for (int rows = 1; rows <= 32; ++rows) {
        const long long blocks = (batch + rows - 1) / rows * (long long)across;
        const long long time = (blocks + at_once - 1) / at_once * (rows + 1);
        if (time < least) {
            least = time;
            best = rows;
        }
    }
    return best;
}

int scan_mark_tile();   // tokens of a tile of the backward's marks; a segment is whole tiles
cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanArgs &a, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs &a, int batch, cudaStream_t s);

struct NormArgs {
    long long R;
    int D, f32, res;          // res: -1 none, else the stream's GDN_DTYPE_*
    int gate;                 // GDN_GATE_*
    float eps, offset, per_d; // per_d: 1 / D
    const void *x, *residual; // forward: the branch and the stream; backward: x for dscale, or null
    const float *scale, *w;   // [D]; scale or null
    const void *z;            // or null
    void *y, *h;
    const void *hin, *dy, *dh;
    void *dx, *dres, *dz;
    float *dw, *dscale;       // [D]
    float *part;              // [blocks, 2 or 1, D]
};
// blocks of the backward (they set the size of its workspace)
int norm_bwd_blocks(long long R, int D, int f32);
cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t s);

}  // namespace gdn
