// gdn_mixer_api.cu -- the extern "C" entry points of the short causal convolution, the selective
// scan and the norms: host-side validation (before any launch), the split plan of the scan, carving
// of the caller's workspaces.
#include <math.h>

#include <algorithm>

#include "gdn_host.h"
#include "gdn_mixer.h"

namespace {

using gdn::aligned16;
using gdn::aligned_to;
using gdn::Carver;
using gdn::cuda_status;
using gdn::kAlign;
using gdn::Span;

constexpr int64_t kGrid = 0x7fffffffLL;
constexpr int32_t kChannels = 1 << 30;   // the kernels' indices of channels stay in 32 bits
constexpr int64_t kTokens = (1LL << 31) - 65536;   // as do those of tokens (rows of a step), a tile past the last

gdn_status check_pack(const gdn_pack *p, gdn::PackArgs *a) {
    if (!p || p->num_seqs < 1 || p->total_tokens < 0 || p->total_tokens > kTokens)
        return GDN_ERR_INVALID_ARG;
    if (!p->cu_seqlens_host || !p->cu_seqlens_dev || !aligned_to(p->cu_seqlens_dev, 4) ||
        !aligned_to(p->device_status, 4))
        return GDN_ERR_INVALID_ARG;
    const int32_t *cu = p->cu_seqlens_host;
    if (cu[0] != 0 || (int64_t)cu[p->num_seqs] != p->total_tokens) return GDN_ERR_INVALID_ARG;
    a->cu_sum = gdn::offset_term(0, 0);
    for (int n = 0; n < p->num_seqs; ++n) {
        if (cu[n + 1] < cu[n]) return GDN_ERR_INVALID_ARG;
        a->cu_sum += gdn::offset_term(n + 1, cu[n + 1]);
    }
    a->N = p->num_seqs;
    a->T = (int)p->total_tokens;
    a->cu = p->cu_seqlens_dev;
    a->status = p->device_status;
    return GDN_OK;
}

// What a call writes (the first `outs` spans) meets nothing else of it.
gdn_status check_overlaps(const Span *spans, size_t count, size_t outs) {
    for (size_t i = 0; i < outs; ++i)
        for (size_t j = i + 1; j < count; ++j)
            if (spans[i].meets(spans[j])) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}
template <size_t N>
gdn_status check_overlaps(const Span (&spans)[N], size_t outs) {
    return check_overlaps(spans, N, outs);
}

size_t bytes_of(int dtype) { return dtype == GDN_DTYPE_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == GDN_DTYPE_BF16 || dtype == GDN_DTYPE_F32; }
// bytes from the first element of strided rows to the last one
size_t rows_span(int64_t rows, int64_t stride, int64_t width, int dtype) {
    return rows > 0 ? (size_t)((rows - 1) * stride + width) * bytes_of(dtype) : 0;
}

struct Pool {
    int32_t num_slots;
    const int32_t *indices, *resume;
    int32_t *status;
};

bool pool_ok(const void *pool, const Pool &s) {
    return pool && s.num_slots >= 1 && s.indices && aligned_to(s.indices, 4) && aligned_to(s.resume, 4) &&
           aligned_to(s.status, 4);
}

gdn::SlotArgs slots_of(const Pool *s) {
    return s ? gdn::SlotArgs{s->num_slots, s->indices, s->resume, s->status} : gdn::SlotArgs{};
}

// ------------------------------------------------------------------------------ convolution
gdn_status check_conv(int32_t channels, int32_t width, int32_t activation, int32_t dtype, int64_t x_stride) {
    if (channels < 1 || channels > kChannels || x_stride < channels || x_stride > ((int64_t)1 << 31)) return GDN_ERR_INVALID_ARG;
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
    if (!known(dtype)) return GDN_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn::ConvArgs conv_args(const gdn::PackArgs &pack, int32_t channels, int32_t width, int32_t activation,
                        int32_t dtype, const void *x, int64_t x_stride, const float *weight,
                        const float *bias) {
    gdn::ConvArgs a{};
    a.pack = pack;
    a.C = channels;
    a.W = width;
    a.silu = activation == GDN_ACT_SILU;
    a.f32 = dtype == GDN_DTYPE_F32;
    a.x = x;
    a.x_stride = x_stride;
    a.w = weight;
    a.bias = bias;
    return a;
}

// Blocks of 128 threads, one channel each, for the tokens' tiles of 8 at least and the sequences.
bool conv_grid_fits(const gdn::PackArgs &p, int32_t channels) {
    const int64_t across = ((int64_t)channels + 127) / 128;
    return (((int64_t)p.T + 7) / 8 + p.N) * across < kGrid;
}

gdn_status conv_fwd(const gdn_pack *p, int32_t channels, int32_t width, int32_t activation, int32_t dtype,
                    const void *x, int64_t x_stride, const float *weight, const float *bias, const void *s0,
                    void *y, void *s1, const Pool *pool, gdn_stream_t stream) {
    gdn::PackArgs pack;
    gdn_status st = check_pack(p, &pack);
    if (st != GDN_OK) return st;
    if ((st = check_conv(channels, width, activation, dtype, x_stride)) != GDN_OK) return st;
    const size_t e = bytes_of(dtype), state = (size_t)channels * (width - 1) * e;
    if (pack.T > 0 && (!x || !y)) return GDN_ERR_INVALID_ARG;
    if (!weight || !aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(x, e) || !aligned16(y) ||
        !aligned16(s0) || !aligned16(s1))
        return GDN_ERR_INVALID_ARG;
    if (pool && !pool_ok(s1, *pool)) return GDN_ERR_INVALID_ARG;
    if (!conv_grid_fits(pack, channels)) return GDN_ERR_INVALID_ARG;
    const size_t each = pack.N * sizeof(int32_t);
    const Span spans[] = {{y, (size_t)pack.T * channels * e},
                          {s1, state * (pool ? pool->num_slots : pack.N)},
                          {x, rows_span(pack.T, x_stride, channels, dtype)},
                          {weight, sizeof(float) * channels * width}, {bias, sizeof(float) * channels},
                          {pool ? nullptr : s0, state * pack.N}, {pack.cu, each + sizeof(int32_t)},
                          {pack.status, sizeof(int32_t)}, {pool ? pool->indices : nullptr, each},
                          {pool ? pool->resume : nullptr, each}, {pool ? pool->status : nullptr, sizeof(int32_t)}};
    if ((st = check_overlaps(spans, 2)) != GDN_OK) return st;
    gdn::ConvArgs a = conv_args(pack, channels, width, activation, dtype, x, x_stride, weight, bias);
    a.slots = slots_of(pool);
    a.s0 = s0;
    a.s1 = s1;
    a.y = y;
    return cuda_status(gdn::launch_conv_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

int conv_tiles(const gdn::PackArgs &p) {
    return (int)(((int64_t)p.T + gdn::conv_bwd_tile() - 1) / gdn::conv_bwd_tile());
}

size_t conv_workspace(const gdn::PackArgs &p, int32_t channels, int32_t width) {
    Carver c(nullptr);
    c.take<float>(std::max<size_t>(1, (size_t)conv_tiles(p) * channels * (width + 1)));
    return c.used();
}

// ------------------------------------------------------------------------------ scan
struct ScanWidth {
    int64_t xs, dts, zs, bs, cs;
};

gdn_status check_scan(const gdn_scan_shape *s, ScanWidth *w) {
    if (!s || s->channels < 1 || s->channels > kChannels || s->groups < 1 || s->groups > s->channels || !known(s->dtype) ||
        s->segment_tokens < -1)
        return GDN_ERR_INVALID_ARG;
    if (s->channels % s->groups != 0) return GDN_ERR_UNSUPPORTED;
    if (s->state_dim != 8 && s->state_dim != 16 && s->state_dim != 32) return GDN_ERR_UNSUPPORTED;
    const int64_t C = s->channels, R = (int64_t)s->groups * s->state_dim;
    *w = {s->x_stride ? s->x_stride : C, s->dt_stride ? s->dt_stride : C, s->z_stride ? s->z_stride : C,
          s->b_stride ? s->b_stride : R, s->c_stride ? s->c_stride : R};
    const int64_t most = (int64_t)1 << 31;
    if (w->xs < C || w->dts < C || w->zs < C || w->bs < R || w->cs < R || w->xs > most || w->dts > most ||
        w->zs > most || w->bs > most || w->cs > most)
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Blocks of a segment; a block's channels are the kernels' (forward: 128 threads of up to 16 states).
int scan_block(const gdn_scan_shape *s, int for_backward) {
    return for_backward ? 1024 / s->state_dim : s->state_dim == 32 ? 64 : 128;
}
int64_t scan_across(const gdn_scan_shape *s, int for_backward) {
    const int64_t per = s->channels / s->groups, cb = scan_block(s, for_backward);
    return s->groups * ((per + cb - 1) / cb);
}

constexpr int kSegment = 32;   // segments are whole tiles of every kernel that walks them
constexpr int kNoSplit = 0x7fffffff;

// Tokens of a segment (kNoSplit: none).  A block walks its tokens one after another, so a few long sequences
// leave SMs idle, and blocks of one length end together, or one wave of them late.  Times are in units of a
// token's in a block that has its SM for itself (forward 90 ns, backward 260 ns); a second block on an SM
// makes it worth 1.08 or 1.27.  A split walk takes as long as its blocks' tokens over the SMs (a segment's
// pipeline fills and drains in 24 or 32), half a segment for the last ones, 70 or 60 for the launches and
// one for each segment of the longest sequence, whose records are joined one after another.  A split
// forward walks its segments for their ends first, at 0.66 of a token; the backward walks ahead anyway.
// Measured, unsplit and split: forward of 4 x 4096 tokens of 4096 channels 334 and 473 us, of 65536 of 2048
// 5200 and 917; backward of the same 4 x 4096 1697 and 1635, of 11 sequences up to 6969 tokens 2360 and 1627.
int plan_scan(const gdn_pack *p, const gdn_scan_shape *s, const gdn::PackArgs &pack, int for_backward) {
    if (s->segment_tokens < 0) return kNoSplit;
    if (s->segment_tokens > 0) {
        const int64_t seg = ((int64_t)s->segment_tokens + kSegment - 1) / kSegment * kSegment;
        return seg <= pack.T ? (int)seg : kNoSplit;
    }
    const int32_t *cu = p->cu_seqlens_host;
    const double across = (double)scan_across(s, for_backward), blocks = across * pack.N;
    const double each = pack.T * across / ((for_backward ? 1.27 : 1.08) * 152.0), fill = for_backward ? 32.0 : 24.0;
    int longest = 0;
    for (int n = 0; n < pack.N; ++n) longest = std::max(longest, cu[n + 1] - cu[n]);
    double best = std::max(1.2 * longest, each);
    if (for_backward) {   // (up to 304 blocks run at once, 1.6 of a token's time each; more of them in waves)
        const double waves = blocks <= 152 ? 0.0 : blocks <= 304 ? std::min(1.6 * longest, each + 0.5 * longest) : each + 0.45 * longest;
        best = std::max(1.05 * longest, waves);
    }
    int seg = kNoSplit;
    for (int64_t L = kSegment; L < longest; L *= 2) {   // (in 64 bits: sequences may be longer than 2^30)
        const double bytes = 4.0 * (pack.N + pack.T / L) * s->channels * (2.0 * s->state_dim + 1.0);
        if (bytes > 1073741824.0) continue;
        auto walk = [&](double part) { return std::max((double)L, part * each * (1.0 + fill / L) + 0.5 * L); };
        double t = walk(1.0) + (for_backward ? 60.0 : 70.0) + longest / L;
        if (!for_backward) {
            double ends = 0.0;   // the tokens ahead of sequences' last segments
            for (int n = 0; n < pack.N; ++n) {
                const int len = cu[n + 1] - cu[n];
                ends += len > 0 ? (double)((len - 1) / L * L) : 0.0;
            }
            t += 0.66 * walk(ends / std::max(1, pack.T));
        }
        if (t < best) {
            best = t;
            seg = (int)L;   // (less than the longest sequence)
        }
    }
    return seg;
}

size_t carve_scan(const gdn_scan_shape *s, gdn::ScanArgs &a, int for_backward, void *workspace) {
    Carver c(workspace);
    const size_t items = (size_t)gdn::scan_items(a.pack.N, a.pack.T, a.seg), C = s->channels, NS = s->state_dim;
    if (a.seg <= a.pack.T) {
        a.rec_h = c.take<float>(items * C * NS);
        a.rec_d = c.take<float>(items * C);
        if (for_backward) a.rec_g = c.take<float>(items * C * NS);
    }
    if (for_backward) {
        const size_t per = C / s->groups, blocks = (per + scan_block(s, 1) - 1) / scan_block(s, 1);
        const size_t marks = (size_t)a.pack.N + a.pack.T / gdn::scan_mark_tile();
        a.marks = c.take<float>(marks * C * NS);
        if (a.seg <= a.pack.T) a.mark_d = c.take<float>(marks * C);
        a.part_bc = c.take<float>(blocks * (size_t)a.pack.T * s->groups * 2 * NS);
        a.part_c = c.take<float>(items * C * (NS + 2));
    }
    return c.used();
}

bool scan_grid_fits(const gdn_scan_shape *s, const gdn::ScanArgs &a) {
    const int64_t bc = (int64_t)a.pack.T * s->groups * s->state_dim / 512, par = (int64_t)s->channels * 34 / 32;
    const int64_t join = ((int64_t)s->channels * s->state_dim / 512 + 1) * a.pack.N;
    return (gdn::scan_items(a.pack.N, a.pack.T, a.seg) + 1) * scan_across(s, 1) < kGrid && bc + 1 < kGrid && par + 1 < kGrid && join < kGrid;
}

gdn::ScanArgs scan_args(const gdn::PackArgs &pack, const gdn_scan_shape *s, const ScanWidth &w, const void *x,
                        const void *dt, const float *A_log, const void *B, const void *C, const float *D,
                        const void *z, const float *dt_bias) {
    gdn::ScanArgs a{};
    a.pack = pack;
    a.C = s->channels;
    a.G = s->groups;
    a.Ns = s->state_dim;
    a.f32 = s->dtype == GDN_DTYPE_F32;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.B = B;
    a.Cm = C;
    a.xs = w.xs;
    a.dts = w.dts;
    a.zs = w.zs;
    a.bs = w.bs;
    a.cs = w.cs;
    a.A_log = A_log;
    a.D = D;
    a.dt_bias = dt_bias;
    a.seg = kNoSplit;
    return a;
}

// The inputs that every form has.
gdn_status check_scan_inputs(const gdn_scan_shape *s, int64_t rows, const void *x, const void *dt,
                             const float *A_log, const void *B, const void *C, const float *D,
                             const void *z, const float *dt_bias) {
    const size_t e = bytes_of(s->dtype);
    if (rows > 0 && (!x || !dt || !B || !C)) return GDN_ERR_INVALID_ARG;
    if (!A_log || !aligned_to(A_log, 4) || !aligned_to(D, 4) || !aligned_to(dt_bias, 4)) return GDN_ERR_INVALID_ARG;
    const void *rows_of[] = {x, dt, z, B, C};
    for (const void *p : rows_of)
        if (!aligned_to(p, e)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Their spans, for the overlap checks.
constexpr size_t kScanInputs = 8;
void scan_spans(const gdn_scan_shape *s, const ScanWidth &w, int64_t rows, const gdn::ScanArgs &a, Span *out) {
    const int64_t R = (int64_t)s->groups * s->state_dim;
    const Span spans[kScanInputs] = {{a.x, rows_span(rows, w.xs, s->channels, s->dtype)},
                                     {a.dt, rows_span(rows, w.dts, s->channels, s->dtype)},
                                     {a.z, rows_span(rows, w.zs, s->channels, s->dtype)},
                                     {a.B, rows_span(rows, w.bs, R, s->dtype)},
                                     {a.Cm, rows_span(rows, w.cs, R, s->dtype)},
                                     {a.A_log, sizeof(float) * s->channels * s->state_dim},
                                     {a.D, sizeof(float) * s->channels}, {a.dt_bias, sizeof(float) * s->channels}};
    std::copy(spans, spans + kScanInputs, out);
}

gdn_status check_workspace(size_t need, bool optional, void *workspace, size_t ws_size) {
    if (optional && !workspace && ws_size == 0) return need > 0 ? GDN_ERR_WORKSPACE_TOO_SMALL : GDN_OK;
    if (!workspace || !aligned_to(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    return ws_size < need ? GDN_ERR_WORKSPACE_TOO_SMALL : GDN_OK;
}

gdn_status scan_fwd(const gdn_pack *p, const gdn_scan_shape *s, const void *x, const void *dt, const float *A_log,
                    const void *B, const void *C, const float *D, const void *z, const float *dt_bias,
                    const float *s0, void *y, float *s1, const Pool *pool, void *workspace, size_t ws_size,
                    gdn_stream_t stream) {
    gdn::PackArgs pack;
    ScanWidth w;
    gdn_status st = check_pack(p, &pack);
    if (st != GDN_OK) return st;
    if ((st = check_scan(s, &w)) != GDN_OK) return st;
    if ((st = check_scan_inputs(s, pack.T, x, dt, A_log, B, C, D, z, dt_bias)) != GDN_OK) return st;
    if ((pack.T > 0 && !y) || !aligned16(y) || !aligned16(s0) || !aligned16(s1)) return GDN_ERR_INVALID_ARG;
    if (pool && !pool_ok(s1, *pool)) return GDN_ERR_INVALID_ARG;
    gdn::ScanArgs a = scan_args(pack, s, w, x, dt, A_log, B, C, D, z, dt_bias);
    a.slots = slots_of(pool);
    a.s0 = s0;
    a.s1 = s1;
    a.y = y;
    a.seg = plan_scan(p, s, pack, 0);
    if (!scan_grid_fits(s, a)) return GDN_ERR_INVALID_ARG;
    const size_t need = carve_scan(s, a, 0, workspace);
    if ((st = check_workspace(need, true, workspace, ws_size)) != GDN_OK) return st;
    const size_t state = sizeof(float) * s->channels * s->state_dim, each = pack.N * sizeof(int32_t);
    Span spans[3 + kScanInputs + 6] = {{y, rows_span(pack.T, s->channels, s->channels, s->dtype)},
                                       {s1, state * (pool ? pool->num_slots : pack.N)}, {workspace, need}};
    scan_spans(s, w, pack.T, a, spans + 3);
    const Span rest[6] = {{pool ? nullptr : s0, state * pack.N}, {pack.cu, each + sizeof(int32_t)},
                          {pack.status, sizeof(int32_t)}, {pool ? pool->indices : nullptr, each},
                          {pool ? pool->resume : nullptr, each}, {pool ? pool->status : nullptr, sizeof(int32_t)}};
    std::copy(rest, rest + 6, spans + 3 + kScanInputs);
    if ((st = check_overlaps(spans, 3)) != GDN_OK) return st;
    return cuda_status(gdn::launch_scan_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------------------ norm
gdn_status check_norm(int64_t rows, int32_t dim, int32_t dtype, int32_t residual_dtype, int32_t gate, float eps,
                      float offset, const float *scale, const float *weight, const void *z) {
    if (rows < 0 || dim < 1 || !known(dtype) || !(eps >= 0.f) || !isfinite(eps) || !isfinite(offset))
        return GDN_ERR_INVALID_ARG;
    if (dim > 8192) return GDN_ERR_UNSUPPORTED;
    if (rows > ((int64_t)1 << 30)) return GDN_ERR_INVALID_ARG;
    if (residual_dtype != GDN_NO_RESIDUAL && !known(residual_dtype)) return GDN_ERR_INVALID_ARG;
    if (dtype == GDN_DTYPE_F32 && residual_dtype == GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
    if (gate != GDN_GATE_NONE && gate != GDN_GATE_SILU && gate != GDN_GATE_SIGMOID) return GDN_ERR_INVALID_ARG;
    if (residual_dtype == GDN_NO_RESIDUAL && scale) return GDN_ERR_INVALID_ARG;
    if (!weight || !aligned16(weight) || !aligned16(scale) || !aligned16(z)) return GDN_ERR_INVALID_ARG;
    if (rows > 0 && (gate != GDN_GATE_NONE) != (z != nullptr)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn::NormArgs norm_args(int64_t rows, int32_t dim, int32_t dtype, int32_t residual_dtype, int32_t gate, float eps,
                        float offset, const float *scale, const float *weight, const void *z) {
    gdn::NormArgs a{};
    a.R = rows;
    a.D = dim;
    a.f32 = dtype == GDN_DTYPE_F32;
    a.res = residual_dtype;
    a.gate = gate;
    a.eps = eps;
    a.offset = offset;
    a.per_d = 1.f / (float)dim;
    a.scale = scale;
    a.w = weight;
    a.z = z;
    return a;
}

size_t norm_workspace(int64_t rows, int32_t dim, int32_t dtype, bool scale) {
    Carver c(nullptr);
    c.take<float>((size_t)gdn::norm_bwd_blocks(rows, dim, dtype == GDN_DTYPE_F32) * (scale ? 2 : 1) * dim);
    return c.used();
}

}  // namespace

extern "C" {

gdn_status gdn_short_conv_fwd(const gdn_pack *p, int32_t channels, int32_t width, int32_t activation,
                              int32_t dtype, const void *x, int64_t x_stride, const float *weight,
                              const float *bias, const void *initial_state, void *y,
                              void *final_state, gdn_stream_t stream) {
    return conv_fwd(p, channels, width, activation, dtype, x, x_stride, weight, bias, initial_state, y, final_state,
                    nullptr, stream);
}

gdn_status gdn_short_conv_prefill_paged(const gdn_pack *p, int32_t channels, int32_t width,
                                        int32_t activation, int32_t dtype, const void *x,
                                        int64_t x_stride, const float *weight, const float *bias,
                                        void *conv_pool, int32_t num_slots,
                                        const int32_t *state_indices,
                                        const int32_t *has_initial_state, void *y,
                                        int32_t *device_status, gdn_stream_t stream) {
    const Pool pool{num_slots, state_indices, has_initial_state, device_status};
    return conv_fwd(p, channels, width, activation, dtype, x, x_stride, weight, bias, conv_pool, y, conv_pool, &pool,
                    stream);
}

size_t gdn_short_conv_workspace_bytes(const gdn_pack *p, int32_t channels, int32_t width) {
    gdn::PackArgs pack;
    if (check_pack(p, &pack) != GDN_OK || channels < 1 || channels > kChannels || width < 2 || width > 4) return 0;
    return conv_workspace(pack, channels, width);
}

gdn_status gdn_short_conv_bwd(const gdn_pack *p, int32_t channels, int32_t width, int32_t activation,
                              int32_t dtype, const void *x, int64_t x_stride, const float *weight,
                              const float *bias, const void *initial_state, const void *d_y,
                              const void *d_final_state, void *dx, float *dweight, float *dbias,
                              void *d_initial_state, void *workspace, size_t ws_size,
                              gdn_stream_t stream) {
    gdn::PackArgs pack;
    gdn_status st = check_pack(p, &pack);
    if (st != GDN_OK) return st;
    if ((st = check_conv(channels, width, activation, dtype, x_stride)) != GDN_OK) return st;
    const size_t e = bytes_of(dtype), state = (size_t)channels * (width - 1) * e * pack.N;
    if (pack.T > 0 && (!x || !d_y || !dx)) return GDN_ERR_INVALID_ARG;
    if (!weight || !dweight || !aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(dweight, 4) ||
        !aligned_to(dbias, 4) || !aligned_to(x, e))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {initial_state, d_y, d_final_state, dx, d_initial_state};
    for (const void *q : ptrs)
        if (!aligned16(q)) return GDN_ERR_INVALID_ARG;
    if (!conv_grid_fits(pack, channels)) return GDN_ERR_INVALID_ARG;
    const size_t need = conv_workspace(pack, channels, width);
    if ((st = check_workspace(need, false, workspace, ws_size)) != GDN_OK) return st;
    const size_t tokens = (size_t)pack.T * channels * e, weights = sizeof(float) * channels * width;
    const Span spans[] = {{dx, tokens}, {dweight, weights}, {dbias, sizeof(float) * channels},
                          {d_initial_state, state}, {workspace, need},
                          {x, rows_span(pack.T, x_stride, channels, dtype)}, {weight, weights},
                          {bias, sizeof(float) * channels}, {initial_state, state}, {d_y, tokens},
                          {d_final_state, state}, {pack.cu, (pack.N + 1) * sizeof(int32_t)},
                          {pack.status, sizeof(int32_t)}};
    if ((st = check_overlaps(spans, 5)) != GDN_OK) return st;
    gdn::ConvArgs a = conv_args(pack, channels, width, activation, dtype, x, x_stride, weight, bias);
    a.s0 = initial_state;
    a.dy = d_y;
    a.ds1 = d_final_state;
    a.dx = dx;
    a.dw = dweight;
    a.dbias = dbias;
    a.ds0 = d_initial_state;
    a.part = static_cast<float *>(workspace);
    a.tile = gdn::conv_bwd_tile();
    a.tiles = conv_tiles(pack);
    return cuda_status(gdn::launch_conv_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_short_conv_step(int32_t batch, int32_t channels, int32_t width, int32_t activation,
                               int32_t dtype, const void *x, int64_t x_stride, const float *weight,
                               const float *bias, void *conv_pool, int32_t num_slots,
                               const int32_t *state_indices, void *y, int32_t *device_status,
                               gdn_stream_t stream) {
    if (batch < 0 || batch > kTokens) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_conv(channels, width, activation, dtype, x_stride);
    if (st != GDN_OK) return st;
    const Pool pool{num_slots, state_indices, nullptr, device_status};
    if (num_slots < 1 || (int64_t)batch * (((int64_t)channels + 127) / 128) > kGrid) return GDN_ERR_INVALID_ARG;
    if (batch == 0) return GDN_OK;
    const size_t e = bytes_of(dtype);
    if (!x || !y || !weight || !pool_ok(conv_pool, pool)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(x, e) || !aligned16(y) || !aligned16(conv_pool))
        return GDN_ERR_INVALID_ARG;
    const Span spans[] = {{y, (size_t)batch * channels * e},
                          {conv_pool, (size_t)num_slots * channels * (width - 1) * e},
                          {x, rows_span(batch, x_stride, channels, dtype)},
                          {weight, sizeof(float) * channels * width}, {bias, sizeof(float) * channels},
                          {state_indices, batch * sizeof(int32_t)}, {device_status, sizeof(int32_t)}};
    if ((st = check_overlaps(spans, 2)) != GDN_OK) return st;
    gdn::PackArgs pack{};
    pack.N = pack.T = batch;
    gdn::ConvArgs a = conv_args(pack, channels, width, activation, dtype, x, x_stride, weight, bias);
    a.slots = slots_of(&pool);
    a.s1 = conv_pool;
    a.y = y;
    return cuda_status(gdn::launch_conv_step(a, batch, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdn_selective_scan_workspace_bytes(const gdn_pack *p, const gdn_scan_shape *s, int for_backward) {
    gdn::PackArgs pack;
    ScanWidth w;
    if (for_backward < 0 || for_backward > 1 || check_pack(p, &pack) != GDN_OK || check_scan(s, &w) != GDN_OK) return 0;
    gdn::ScanArgs a{};
    a.pack = pack;
    a.seg = plan_scan(p, s, pack, for_backward);
    return std::max(kAlign, carve_scan(s, a, for_backward, nullptr));
}

gdn_status gdn_selective_scan_fwd(const gdn_pack *p, const gdn_scan_shape *s, const void *x,
                                  const void *dt, const float *A_log, const void *B, const void *C,
                                  const float *D, const void *z, const float *dt_bias,
                                  const float *initial_state, void *y, float *final_state,
                                  void *workspace, size_t ws_size, gdn_stream_t stream) {
    return scan_fwd(p, s, x, dt, A_log, B, C, D, z, dt_bias, initial_state, y, final_state, nullptr, workspace, ws_size,
                    stream);
}

gdn_status gdn_selective_scan_prefill_paged(const gdn_pack *p, const gdn_scan_shape *s,
                                            const void *x, const void *dt, const float *A_log,
                                            const void *B, const void *C, const float *D,
                                            const void *z, const float *dt_bias, float *state_pool,
                                            int32_t num_slots, const int32_t *state_indices,
                                            const int32_t *has_initial_state, void *y,
                                            int32_t *device_status, void *workspace,
                                            size_t ws_size, gdn_stream_t stream) {
    const Pool pool{num_slots, state_indices, has_initial_state, device_status};
    return scan_fwd(p, s, x, dt, A_log, B, C, D, z, dt_bias, state_pool, y, state_pool, &pool, workspace, ws_size,
                    stream);
}

gdn_status gdn_selective_scan_bwd(const gdn_pack *p, const gdn_scan_shape *s, const void *x,
                                  const void *dt, const float *A_log, const void *B, const void *C,
                                  const float *D, const void *z, const float *dt_bias,
                                  const float *initial_state, const void *d_y,
                                  const float *d_final_state, void *dx, void *ddt, float *dA_log,
                                  void *dB, void *dC, float *dD, void *dz, float *ddt_bias,
                                  float *d_initial_state, void *workspace, size_t ws_size,
                                  gdn_stream_t stream) {
    gdn::PackArgs pack;
    ScanWidth w;
    gdn_status st = check_pack(p, &pack);
    if (st != GDN_OK) return st;
    if ((st = check_scan(s, &w)) != GDN_OK) return st;
    if ((st = check_scan_inputs(s, pack.T, x, dt, A_log, B, C, D, z, dt_bias)) != GDN_OK) return st;
    if (pack.T > 0 && (!d_y || !dx || !ddt || !dB || !dC || (z != nullptr) != (dz != nullptr))) return GDN_ERR_INVALID_ARG;
    if (!dA_log || !aligned_to(dA_log, 4) || !aligned_to(dD, 4) || !aligned_to(ddt_bias, 4)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {initial_state, d_y, d_final_state, dx, ddt, dB, dC, dz, d_initial_state};
    for (const void *q : ptrs)
        if (!aligned16(q)) return GDN_ERR_INVALID_ARG;
    gdn::ScanArgs a = scan_args(pack, s, w, x, dt, A_log, B, C, D, z, dt_bias);
    a.s0 = initial_state;
    a.dy = d_y;
    a.ds1 = d_final_state;
    a.dx = dx;
    a.ddt = ddt;
    a.dz = dz;
    a.dB = dB;
    a.dC = dC;
    a.dA_log = dA_log;
    a.dD = dD;
    a.ddt_bias = ddt_bias;
    a.ds0 = d_initial_state;
    a.seg = plan_scan(p, s, pack, 1);
    if (!scan_grid_fits(s, a)) return GDN_ERR_INVALID_ARG;
    const size_t need = carve_scan(s, a, 1, workspace);
    if ((st = check_workspace(need, false, workspace, ws_size)) != GDN_OK) return st;
    const size_t tokens = rows_span(pack.T, s->channels, s->channels, s->dtype);
    const int64_t R = (int64_t)s->groups * s->state_dim;
    const size_t rows = rows_span(pack.T, R, R, s->dtype), par = sizeof(float) * s->channels;
    const size_t state = par * s->state_dim * pack.N;
    Span spans[10 + kScanInputs + 5] = {{dx, tokens}, {ddt, tokens}, {dz, tokens}, {dB, rows}, {dC, rows},
                                        {dA_log, par * s->state_dim}, {dD, par}, {ddt_bias, par},
                                        {d_initial_state, state}, {workspace, need}};
    scan_spans(s, w, pack.T, a, spans + 10);
    const Span rest[5] = {{initial_state, state}, {d_y, tokens}, {d_final_state, state},
                          {pack.cu, (pack.N + 1) * sizeof(int32_t)}, {pack.status, sizeof(int32_t)}};
    std::copy(rest, rest + 5, spans + 10 + kScanInputs);
    if ((st = check_overlaps(spans, 10)) != GDN_OK) return st;
    return cuda_status(gdn::launch_scan_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_selective_scan_step(int32_t batch, const gdn_scan_shape *s, const void *x,
                                   const void *dt, const float *A_log, const void *B,
                                   const void *C, const float *D, const void *z,
                                   const float *dt_bias, float *state_pool, int32_t num_slots,
                                   const int32_t *state_indices, void *y, int32_t *device_status,
                                   gdn_stream_t stream) {
    ScanWidth w;
    if (batch < 0 || batch > kTokens) return GDN_ERR_INVALID_ARG;
    gdn_status st = check_scan(s, &w);
    if (st != GDN_OK) return st;
    if (num_slots < 1 || (int64_t)batch * (((int64_t)s->channels + 31) / 32) > kGrid) return GDN_ERR_INVALID_ARG;
    if (batch == 0) return GDN_OK;
    if ((st = check_scan_inputs(s, batch, x, dt, A_log, B, C, D, z, dt_bias)) != GDN_OK) return st;
    const Pool pool{num_slots, state_indices, nullptr, device_status};
    if (!y || !pool_ok(state_pool, pool) || !aligned16(y) || !aligned16(state_pool)) return GDN_ERR_INVALID_ARG;
    gdn::PackArgs pack{};
    pack.N = pack.T = batch;
    gdn::ScanArgs a = scan_args(pack, s, w, x, dt, A_log, B, C, D, z, dt_bias);
    a.slots = slots_of(&pool);
    a.s1 = state_pool;
    a.y = y;
    Span spans[2 + kScanInputs + 2] = {{y, rows_span(batch, s->channels, s->channels, s->dtype)},
                                       {state_pool, sizeof(float) * s->channels * s->state_dim * num_slots}};
    scan_spans(s, w, batch, a, spans + 2);
    spans[2 + kScanInputs] = {state_indices, batch * sizeof(int32_t)};
    spans[3 + kScanInputs] = {device_status, sizeof(int32_t)};
    if ((st = check_overlaps(spans, 2)) != GDN_OK) return st;
    return cuda_status(gdn::launch_scan_step(a, batch, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_rms_norm_fwd(int64_t rows, int32_t dim, int32_t dtype, int32_t residual_dtype,
                            int32_t gate, float eps, float offset, const void *x,
                            const void *residual, const float *scale, const float *weight,
                            const void *z, void *y, void *h, gdn_stream_t stream) {
    gdn_status st = check_norm(rows, dim, dtype, residual_dtype, gate, eps, offset, scale, weight, z);
    if (st != GDN_OK) return st;
    const bool stream_there = residual_dtype != GDN_NO_RESIDUAL;
    if (rows == 0) return GDN_OK;
    if (!x || !y || stream_there != (residual != nullptr) || stream_there != (h != nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(y) || !aligned16(h)) return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * dim, e = bytes_of(dtype), r = stream_there ? bytes_of(residual_dtype) : 0;
    const Span spans[] = {{y, n * e}, {h, n * r}, {x, n * e}, {residual, n * r}, {z, n * e},
                          {scale, sizeof(float) * dim}, {weight, sizeof(float) * dim}};
    if ((st = check_overlaps(spans, 2)) != GDN_OK) return st;
    gdn::NormArgs a = norm_args(rows, dim, dtype, residual_dtype, gate, eps, offset, scale, weight, z);
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.h = h;
    return cuda_status(gdn::launch_norm_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdn_rms_norm_workspace_bytes(int64_t rows, int32_t dim, int32_t dtype, int32_t with_scale) {
    if (rows < 0 || rows > ((int64_t)1 << 30) || dim < 1 || dim > 8192 || !known(dtype)) return 0;
    return norm_workspace(rows, dim, dtype, with_scale != 0);
}

gdn_status gdn_rms_norm_bwd(int64_t rows, int32_t dim, int32_t dtype, int32_t residual_dtype,
                            int32_t gate, float eps, float offset, const void *h, const void *x,
                            const float *scale, const float *weight, const void *z,
                            const void *d_y, const void *d_h, void *dx, void *dresidual, void *dz,
                            float *dweight, float *dscale, void *workspace, size_t ws_size,
                            gdn_stream_t stream) {
    gdn_status st = check_norm(rows, dim, dtype, residual_dtype, gate, eps, offset, scale, weight, z);
    if (st != GDN_OK) return st;
    const bool stream_there = residual_dtype != GDN_NO_RESIDUAL;
    if (rows > 0 && (!h || !d_y || !dx || (z != nullptr) != (dz != nullptr) || (scale != nullptr) != (x != nullptr)))
        return GDN_ERR_INVALID_ARG;
    if (!dweight || (scale != nullptr) != (dscale != nullptr)) return GDN_ERR_INVALID_ARG;
    if (!stream_there && (d_h || dresidual)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {h, x, d_y, d_h, dx, dresidual, dz};
    for (const void *q : ptrs)
        if (!aligned16(q)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(dweight, 4) || !aligned_to(dscale, 4)) return GDN_ERR_INVALID_ARG;
    const size_t need = norm_workspace(rows, dim, dtype, scale != nullptr);
    if ((st = check_workspace(need, false, workspace, ws_size)) != GDN_OK) return st;
    const size_t n = (size_t)rows * dim, e = bytes_of(dtype), r = stream_there ? bytes_of(residual_dtype) : e;
    const size_t par = sizeof(float) * dim;
    const Span spans[] = {{dx, n * e}, {dresidual, n * r}, {dz, n * e}, {dweight, par}, {dscale, par}, {workspace, need},
                          {h, n * r}, {x, n * e}, {d_y, n * e}, {d_h, n * r}, {z, n * e}, {scale, par}, {weight, par}};
    if ((st = check_overlaps(spans, 6)) != GDN_OK) return st;
    gdn::NormArgs a = norm_args(rows, dim, dtype, residual_dtype, gate, eps, offset, scale, weight, z);
    a.hin = h;
    a.x = x;
    a.dy = d_y;
    a.dh = d_h;
    a.dx = dx;
    a.dres = dresidual;
    a.dz = dz;
    a.dw = dweight;
    a.dscale = dscale;
    a.part = static_cast<float *>(workspace);
    return cuda_status(gdn::launch_norm_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
