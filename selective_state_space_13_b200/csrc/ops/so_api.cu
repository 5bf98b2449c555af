// Host entry points of the operators around the scan (the C ABI of include/selective_scan_ops.h):
// argument validation, workspace plans and launches.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "so_internal.h"
#include "ss_internal.h"

namespace {

constexpr int64_t kMaxI32 = (int64_t{1} << 31) - 1;
constexpr int kMaxSegments = 1024;
// Rows of a call with a list of slots that must not repeat: every row looks through the list before it,
// so that the look-ups grow with the square of the rows (2^20 of them: by estimate 0.2 s a channel tile).
constexpr int64_t kMostListedRows = int64_t{1} << 20;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(std::initializer_list<const void*> ps, size_t a)
{
    for (const void* p : ps)
        if (p && reinterpret_cast<uintptr_t>(p) % a)
            return false;
    return true;
}

// The limits of selective_scan_fwd on sizes, types and the row pitch.
ss_status check_shape(const ss_shape* s)
{
    if (!s)
        return SS_ERR_NULL;
    if (s->reserved != 0)
        return SS_ERR_SHAPE;
    if (s->io_dtype != SS_F32 && s->io_dtype != SS_BF16)
        return SS_ERR_DTYPE;
    if (s->batch < 0 || s->seqlen < 0 || s->dim < 0 || s->dstate < 1 || s->seqlen > kMaxI32 ||
        s->batch > (int64_t{1} << 24) || s->dim > (int64_t{1} << 24))
        return SS_ERR_SHAPE;
    if (s->dstate > SS_MAX_DSTATE)
        return SS_ERR_UNSUPPORTED;
    if (s->batch * s->seqlen * SS_MAX_DIRS > kMaxI32 || s->seqlen * s->dim > kMaxI32)
        return SS_ERR_SHAPE;
    if ((s->dim * (s->io_dtype == SS_BF16 ? 2 : 4)) % 16 != 0)
        return SS_ERR_ALIGN;
    return SS_OK;
}

// The stream has to belong to the current device.  While a stream is being captured the runtime
// refuses to say which device it belongs to (and the question would end the capture): it is not
// checked then, and a foreign stream is left to the launches to refuse.
ss_status check_stream(cudaStream_t st)
{
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cap) != cudaSuccess)
        return SS_ERR_CUDA;
    if (cap != cudaStreamCaptureStatusNone)
        return SS_OK;
    int dev = 0, sdev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaStreamGetDevice(st, &sdev) != cudaSuccess)
        return SS_ERR_CUDA;
    return dev == sdev ? SS_OK : SS_ERR_DEVICE;
}

ss_status status_of(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ERR_CUDA; }

// ---------------------------------------------------------------- gated linear recurrence

struct RecPlan {
    int cluster, S;
    int64_t seg_len;
    size_t off_maps, bytes;
};

// CTAs in the cluster of a column of 64 channels.  A B200 runs about three of the recurrence's CTAs
// on each of its 148 SMs best, so a launch takes as long as its whole waves of 444: the cluster is
// the size that fills them best, an eighth dearer for every CTA more that has to be heard.  Measured at
// 1, 2, 4, 6 and 8 CTAs (us, bf16): 8 x 2048 x 1536 (192 columns) 41.4, 34.9, 38.3, 44.6, 47.3; 16 x 2048
// x 1536: 55.7, 61.9, 69.0, 79.9, 88.4; 16 x 1024 x 1024: 24.1, 30.5, 31.2, 36.1, 41.3; 1 x 32768 x 5120:
// 431, 321, 230, 249, 236; 4 x 8192 x 1536: 111, 87, 64, 77, 71; 3 was slower than its neighbours.
constexpr int64_t kRecSlots = 3 * 148;

int rec_cluster(int64_t columns, int64_t tiles)
{
    int best = 1;
    double most = 0.;
    for (int cs : {1, 2, 4, 6, 8}) {
        if (cs > so::kRecMostCluster || cs > tiles)
            break;
        const double waves = static_cast<double>(columns) * cs / kRecSlots;
        const double full = waves / static_cast<double>(ceil_div(columns * cs, kRecSlots));
        const double score = full / (1. + 0.12 * (cs - 1));
        if (score > most) {
            most = score;
            best = cs;
        }
    }
    return best;
}

ss_status plan_recurrence(const ss_shape* s, const ss_recurrence_opts* o, bool backward, RecPlan* pl)
{
    ss_status st = check_shape(s);
    if (st != SS_OK)
        return st;
    if (!o)
        return SS_ERR_NULL;
    if (s->dstate != 1)
        return SS_ERR_SHAPE;
    if ((o->form != SS_GATE_SIGMOID && o->form != SS_GATE_EXP) || o->reserved != 0)
        return SS_ERR_UNSUPPORTED;
    if (o->dir != SS_DIR_FWD && o->dir != SS_DIR_REV)
        return SS_ERR_DIRMAP;
    const int64_t columns = s->batch * ceil_div(s->dim, 64);
    const int64_t tiles = ceil_div(s->seqlen, so::recurrence_tile(s->io_dtype, backward));
    pl->cluster = columns > 0 && tiles > 0 ? rec_cluster(columns, tiles) : 1;
    // Segments only where whole clusters fill less than half of the GPU and a column has rounds to
    // share out: four at least for each segment.
    const int64_t round = static_cast<int64_t>(so::recurrence_tile(s->io_dtype, backward)) * pl->cluster;
    const int64_t rounds = ceil_div(s->seqlen, round);
    int64_t S = 1;
    if (columns > 0 && pl->cluster == so::kRecMostCluster)
        S = kRecSlots / (columns * pl->cluster);
    if (S > rounds / 4)
        S = rounds / 4;
    if (S < 2)
        S = 1;
    pl->seg_len = ceil_div(rounds > 0 ? rounds : 1, S) * round;
    pl->S = static_cast<int>(s->seqlen > 0 ? ceil_div(s->seqlen, pl->seg_len) : 1);
    if (columns * pl->S * pl->cluster > kMaxI32)
        return SS_ERR_SHAPE;
    pl->bytes = 0;
    if (backward && o->form == SS_GATE_SIGMOID)
        pl->bytes = align256(static_cast<size_t>(s->batch) * s->dim * pl->S * pl->cluster *
                             sizeof(float));
    pl->off_maps = pl->bytes;
    if (pl->S > 1)
        pl->bytes += static_cast<size_t>(columns) * pl->S * 32 * sizeof(float4);
    return SS_OK;
}

// ---------------------------------------------------------------- gradient of the scan

struct BwdPlan {
    int K, S;
    bool split;
    int64_t seg_len;
    int32_t dirs[SS_MAX_DIRS];
    int32_t H, W;
    int flags;
    const float* init;
    size_t off_ckpt, off_cum, off_h, off_p, off_g, off_dbc, off_dpar, off_du, off_dz, bytes;
};

// Automatic segments of the gradient.  `units` (direction, batch row, channel tile) CTAs for each
// segment fill the kBwdSlots CTAs that fit on a B200 (3 on each of 148 SMs) in whole waves, so S
// segments take ceil(units S / slots) / S of a whole sequence's time; a step takes 0.7 us, any split
// costs about 15% more work (the segment products, the checkpoints' shift), and every wave folds the
// other segments' states (some 0.47 us for each) and has its ends (5.6 us).  Measured, and from that
// rule: 8 x 2048 x 1536 (192 units) 1434 us unsplit (1434), 923 at S = 2 (831), 752 at 9 (772), 758 at 16
// (813), 795 at 23 (880), 828 at 30 (969); 2 x 333 x 72 in fp32 (4 units) 232 us unsplit (233), 108 at 4
// (74), 70 at 20 (28), 68 at 40 (31): what a call takes besides is not in it; 64 x 197 x 768 in two
// directions (1536 units) 601 us unsplit (552), more with any split.  Its choices are near the best.
constexpr int64_t kBwdSlots = 3 * 148;
constexpr int64_t kBwdMinSteps = 16;
constexpr int64_t kBwdMostAuto = 256;

int64_t bwd_segments(int64_t units, int64_t L)
{
    int64_t best = 1;
    double least = 0.7 * static_cast<double>(L * ceil_div(units, kBwdSlots));
    for (int64_t S = 2; S <= kBwdMostAuto && S <= L / kBwdMinSteps; ++S) {
        const double waves = static_cast<double>(ceil_div(units * S, kBwdSlots));
        const double cost = waves * (0.805 * static_cast<double>(L) / S + 7. / 15. * S + 5.6);
        if (cost < 0.999 * least) {
            least = cost;
            best = S;
        }
    }
    return best;
}

ss_status plan_bwd(const ss_shape* s, const ss_direction_map* dmap, const ss_launch_opts* o,
                   bool gate, BwdPlan* pl)
{
    ss_status st = check_shape(s);
    if (st != SS_OK)
        return st;
    std::memset(pl, 0, sizeof(*pl));
    pl->K = 1;
    if (dmap) {
        if (dmap->num_dirs < 1 || dmap->num_dirs > SS_MAX_DIRS)
            return SS_ERR_DIRMAP;
        pl->K = dmap->num_dirs;
        pl->H = dmap->H;
        pl->W = dmap->W;
        for (int k = 0; k < pl->K; ++k) {
            const int32_t d = dmap->dir[k];
            if (d < SS_DIR_FWD || d > SS_DIR_COL_REV)
                return SS_ERR_DIRMAP;
            pl->dirs[k] = d;
            if ((d == SS_DIR_COL || d == SS_DIR_COL_REV) &&
                (dmap->H <= 0 || dmap->W <= 0 ||
                 static_cast<int64_t>(dmap->H) * dmap->W != s->seqlen))
                return SS_ERR_DIRMAP;
        }
    }
    int64_t want = 0;
    if (o) {
        if (o->reserved != 0 || o->segments < 0 || o->segments > kMaxSegments ||
            (o->flags & ~(SS_FLAG_GENERIC_A | SS_FLAG_U_PER_DIRECTION | SS_FLAG_PARAMS_PER_DIRECTION)) ||
            o->conv_weight || o->conv_bias || o->conv_width != 0 || o->delta_scale ||
            o->scan_begin_event || o->scan_end_event)
            return SS_ERR_UNSUPPORTED;
        pl->flags = o->flags;
        pl->init = o->initial_state;
        want = o->segments;
    }
    const int64_t L = s->seqlen, rows = s->batch * pl->K;
    const int64_t states = s->dstate > 8 ? 16 : 8;  // as the kernels pad them
    const int64_t ctiles = ceil_div(s->dim, so::kBwdCells / states), ntiles = ceil_div(L, so::kBwdTile);
    const int64_t units = rows * ctiles;
    if (want == 0)
        want = bwd_segments(units, L);
    if (want > kMaxSegments)
        want = kMaxSegments;
    if (want > ntiles)
        want = ntiles;
    if (want < 1)
        want = 1;
    pl->seg_len = ntiles > 0 ? ceil_div(ntiles, want) * so::kBwdTile : so::kBwdTile;
    pl->S = L > 0 ? static_cast<int>(ceil_div(L, pl->seg_len)) : 1;
    pl->split = pl->S > 1 || pl->init != nullptr;
    // the blocks of the sweeps and of the launch that adds up what they leave
    if (units * pl->S > kMaxI32 ||
        rows * L / 8 + pl->K * s->dim + 2 * (s->batch * L * s->dim / 1024) + 8 > kMaxI32)
        return SS_ERR_SHAPE;

    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off = align256(off + floats * sizeof(float));
        return at;
    };
    const size_t R = static_cast<size_t>(rows), D = static_cast<size_t>(s->dim);
    pl->off_ckpt = take(R * ntiles * ctiles * so::kBwdCells);
    if (pl->split) {
        pl->off_cum = take(R * ntiles * D);
        const size_t cells = R * pl->S * ctiles * so::kBwdCells;
        pl->off_h = take(cells);
        pl->off_p = take(cells);
        pl->off_g = take(cells);
    }
    pl->off_dbc = take(R * ctiles * L * 2 * states);
    pl->off_dpar = take(R * pl->S * D * (states + 2));
    if (pl->K > 1) {
        const size_t plane = R * L * D;
        if (!(pl->flags & SS_FLAG_U_PER_DIRECTION))
            pl->off_du = take(plane);
        if (gate)
            pl->off_dz = take(plane);
    }
    pl->bytes = off;
    return SS_OK;
}

}  // namespace

extern "C" {

ss_status gated_recurrence_workspace_size(const ss_shape* shape, const ss_recurrence_opts* opts,
                                          int32_t backward, size_t* bytes)
{
    if (!bytes)
        return SS_ERR_NULL;
    RecPlan pl;
    const ss_status st = plan_recurrence(shape, opts, backward != 0, &pl);
    if (st == SS_OK)
        *bytes = pl.bytes;
    return st;
}

ss_status gated_recurrence_fwd(const ss_shape* shape, const ss_recurrence_opts* opts,
                               const void* x, const void* gate, const float* gate_bias,
                               const float* initial_state, void* out, float* last_state,
                               void* workspace, size_t workspace_bytes, void* stream)
{
    RecPlan pl;
    ss_status st = plan_recurrence(shape, opts, false, &pl);
    if (st != SS_OK)
        return st;
    const int64_t b = shape->batch, L = shape->seqlen, D = shape->dim;
    if (opts->form == SS_GATE_EXP && gate_bias)
        return SS_ERR_UNSUPPORTED;
    if (b * L * D > 0 && (!x || !gate || !out))
        return SS_ERR_NULL;
    if (!aligned({x, gate, out, workspace}, 16) ||
        !aligned({gate_bias, initial_state, last_state}, 4))
        return SS_ERR_ALIGN;
    if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes))
        return SS_ERR_WORKSPACE;
    if (b * D == 0)
        return SS_OK;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if ((st = check_stream(strm)) != SS_OK)
        return st;
    if (L == 0) {  // no step is taken: the last state is the initial one
        if (!last_state)
            return SS_OK;
        const size_t n = static_cast<size_t>(b) * D * sizeof(float);
        return status_of(initial_state ? cudaMemcpyAsync(last_state, initial_state, n,
                                                         cudaMemcpyDeviceToDevice, strm)
                                       : cudaMemsetAsync(last_state, 0, n, strm));
    }
    so::RecParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x;
    p.gate = gate;
    p.bias = gate_bias;
    p.init = initial_state;
    p.out = out;
    p.last = last_state;
    p.batch = b;
    p.L = L;
    p.D = D;
    p.cluster = pl.cluster;
    p.S = pl.S;
    p.seg_len = static_cast<int32_t>(pl.seg_len < L ? pl.seg_len : L);
    p.seg_maps = pl.S > 1 ? reinterpret_cast<float4*>(static_cast<unsigned char*>(workspace) +
                                                      pl.off_maps)
                          : nullptr;
    p.form = opts->form;
    p.complement = opts->complement != 0;
    p.reverse = opts->dir == SS_DIR_REV;
    p.status = ss::status_word();
    if (!p.status)
        return SS_ERR_CUDA;
    return status_of(so::launch_recurrence(p, shape->io_dtype, false, strm));
}

ss_status gated_recurrence_bwd(const ss_shape* shape, const ss_recurrence_opts* opts,
                               const void* x, const void* gate, const float* gate_bias,
                               const float* initial_state, const void* out, const void* dout,
                               const float* dlast_state, void* dx, void* dgate,
                               float* dgate_bias, float* dinitial_state, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    RecPlan pl;
    ss_status st = plan_recurrence(shape, opts, true, &pl);
    if (st != SS_OK)
        return st;
    const int64_t b = shape->batch, L = shape->seqlen, D = shape->dim;
    if (opts->form == SS_GATE_EXP && (gate_bias || dgate_bias))
        return SS_ERR_UNSUPPORTED;
    if (b * L * D > 0 && (!x || !gate || !out || !dout || !dx || !dgate))
        return SS_ERR_NULL;
    if (!aligned({x, gate, out, dout, dx, dgate, workspace}, 16) ||
        !aligned({gate_bias, initial_state, dlast_state, dgate_bias, dinitial_state}, 4))
        return SS_ERR_ALIGN;
    if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes))
        return SS_ERR_WORKSPACE;
    if (D == 0)
        return SS_OK;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if ((st = check_stream(strm)) != SS_OK)
        return st;
    if (b * L == 0) {  // no step is taken: the gradient of the last state passes through
        cudaError_t e = cudaSuccess;
        if (dgate_bias)
            e = cudaMemsetAsync(dgate_bias, 0, D * sizeof(float), strm);
        const size_t n = static_cast<size_t>(b) * D * sizeof(float);
        if (e == cudaSuccess && dinitial_state && n > 0)
            e = dlast_state ? cudaMemcpyAsync(dinitial_state, dlast_state, n,
                                              cudaMemcpyDeviceToDevice, strm)
                            : cudaMemsetAsync(dinitial_state, 0, n, strm);
        return status_of(e);
    }
    so::RecParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x;
    p.gate = gate;
    p.bias = gate_bias;
    p.init = initial_state;
    p.out_in = out;
    p.dout = dout;
    p.dlast = dlast_state;
    p.out = dx;
    p.dgate = dgate;
    p.last = dinitial_state;
    p.dbias = dgate_bias;
    p.dbias_part = dgate_bias ? static_cast<float*>(workspace) : nullptr;
    p.batch = b;
    p.L = L;
    p.D = D;
    p.cluster = pl.cluster;
    p.S = pl.S;
    p.seg_len = static_cast<int32_t>(pl.seg_len < L ? pl.seg_len : L);
    p.seg_maps = pl.S > 1 ? reinterpret_cast<float4*>(static_cast<unsigned char*>(workspace) +
                                                      pl.off_maps)
                          : nullptr;
    p.form = opts->form;
    p.complement = opts->complement != 0;
    p.reverse = opts->dir == SS_DIR_REV;
    p.status = ss::status_word();
    if (!p.status)
        return SS_ERR_CUDA;
    return status_of(so::launch_recurrence(p, shape->io_dtype, true, strm));
}

ss_status selective_scan_bwd_workspace_size(const ss_shape* shape, const ss_direction_map* dmap,
                                            const ss_launch_opts* opts, size_t* bytes)
{
    if (!bytes)
        return SS_ERR_NULL;
    BwdPlan pl;
    const ss_status st = plan_bwd(shape, dmap, opts, true, &pl);
    if (st == SS_OK)
        *bytes = pl.bytes;
    return st;
}

ss_status selective_scan_bwd(const ss_shape* shape, const void* u, const void* delta,
                             const float* A, const void* B, const void* C, const float* Dskip,
                             const void* z, const float* delta_bias, int32_t softplus,
                             const ss_direction_map* dmap, const void* dout,
                             const float* dlast_state, const ss_scan_grads* grads,
                             void* workspace, size_t workspace_bytes, void* stream,
                             const ss_launch_opts* opts)
{
    // sized as if there were a gate, so that the answer of the size call holds for both
    BwdPlan pl;
    ss_status st = plan_bwd(shape, dmap, opts, true, &pl);
    if (st != SS_OK)
        return st;
    if (!grads)
        return SS_ERR_NULL;
    const ss_scan_grads& g = *grads;
    const int64_t b = shape->batch, L = shape->seqlen, D = shape->dim, N = shape->dstate;
    const bool has_data = b * L * D > 0;
    if (has_data && (!u || !delta || !B || !C || !dout || !g.du || !g.ddelta || !g.dB || !g.dC))
        return SS_ERR_NULL;
    if (has_data && z && !g.dz)
        return SS_ERR_NULL;
    if (D > 0 && (!A || !g.dA))
        return SS_ERR_NULL;
    if ((!z && g.dz) || (!Dskip && g.dDskip) || (!delta_bias && g.ddelta_bias))
        return SS_ERR_UNSUPPORTED;
    if (!aligned({u, delta, B, C, z, dout, g.du, g.ddelta, g.dB, g.dC, g.dz, workspace}, 16) ||
        !aligned({A, Dskip, delta_bias, pl.init, dlast_state, g.dA, g.dDskip, g.ddelta_bias,
                  g.dinitial_state}, 4))
        return SS_ERR_ALIGN;
    if (has_data && (!workspace || workspace_bytes < pl.bytes))
        return SS_ERR_WORKSPACE;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if ((st = check_stream(strm)) != SS_OK)
        return st;
    if (!has_data) {
        // no step is taken: parameters get zero, the last state's gradient passes through; dB and
        // dC of a call without channels are sums over nothing
        const int64_t sets = (pl.flags & SS_FLAG_PARAMS_PER_DIRECTION) ? pl.K : 1;
        cudaError_t e = cudaSuccess;
        auto zero = [&](void* ptr, int64_t bytes) {
            if (e == cudaSuccess && ptr && bytes > 0)
                e = cudaMemsetAsync(ptr, 0, static_cast<size_t>(bytes), strm);
        };
        const int64_t esz = shape->io_dtype == SS_BF16 ? 2 : 4;
        zero(g.dA, sets * D * N * 4);
        zero(g.dDskip, sets * D * 4);
        zero(g.ddelta_bias, sets * D * 4);
        zero(g.dB, pl.K * b * L * N * esz);
        zero(g.dC, pl.K * b * L * N * esz);
        const int64_t n = pl.K * b * D * N * 4;
        if (!dlast_state)
            zero(g.dinitial_state, n);
        else if (e == cudaSuccess && g.dinitial_state && n > 0)
            e = cudaMemcpyAsync(g.dinitial_state, dlast_state, static_cast<size_t>(n),
                                cudaMemcpyDeviceToDevice, strm);
        return status_of(e);
    }
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    so::BwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.u = u;
    p.delta = delta;
    p.B = B;
    p.C = C;
    p.z = z;
    p.dout = dout;
    p.A = A;
    p.Dskip = Dskip;
    p.bias = delta_bias;
    p.init = pl.init;
    p.dlast = dlast_state;
    p.g = g;
    p.ckpt = at(pl.off_ckpt);
    p.cum = at(pl.off_cum);
    p.seg_h = at(pl.off_h);
    p.seg_p = at(pl.off_p);
    p.seg_g = at(pl.off_g);
    p.dbc = at(pl.off_dbc);
    p.dpar = at(pl.off_dpar);
    p.u_per_dir = (pl.flags & SS_FLAG_U_PER_DIRECTION) ? 1 : 0;
    p.params_per_dir = (pl.flags & SS_FLAG_PARAMS_PER_DIRECTION) ? 1 : 0;
    p.du_part = pl.K > 1 && !p.u_per_dir ? at(pl.off_du) : nullptr;
    p.dz_part = pl.K > 1 && z ? at(pl.off_dz) : nullptr;
    p.batch = b;
    p.L = L;
    p.D = D;
    p.seg_len = pl.seg_len;
    p.N = static_cast<int32_t>(N);
    p.K = pl.K;
    p.S = pl.S;
    for (int k = 0; k < SS_MAX_DIRS; ++k)
        p.dirs[k] = pl.dirs[k];
    p.H = pl.H;
    p.W = pl.W;
    p.softplus = softplus ? 1 : 0;
    if (shape->io_dtype == SS_BF16)
        return status_of(N > 8 ? so::launch_scan_bwd_bf16_4(p, strm)
                               : so::launch_scan_bwd_bf16_2(p, strm));
    return status_of(N > 8 ? so::launch_scan_bwd_f32_4(p, strm) : so::launch_scan_bwd_f32_2(p, strm));
}

ss_status selective_scan_step(const ss_shape* shape, int64_t num_slots, const void* u,
                              const void* delta, const float* A, const void* B, const void* C,
                              const float* Dskip, const void* z, const float* delta_bias,
                              int32_t softplus, float* state, const int32_t* slots,
                              const float* conv_weight, const float* conv_bias,
                              int32_t conv_width, void* conv_state, void* out, void* stream)
{
    ss_status st = check_shape(shape);
    if (st != SS_OK)
        return st;
    const int64_t b = shape->batch, D = shape->dim;
    if (shape->seqlen != 1 || num_slots < 1 || num_slots > kMaxI32 || (!slots && num_slots < b) ||
        (slots && b > kMostListedRows))
        return SS_ERR_SHAPE;
    if (conv_weight ? conv_width < 1 || conv_width > SS_MAX_CONV_WIDTH
                    : conv_width != 0 || conv_bias || conv_state)
        return SS_ERR_UNSUPPORTED;
    if (b * D > 0 && (!u || !delta || !A || !B || !C || !state || !out ||
                      (conv_width > 1 && !conv_state)))
        return SS_ERR_NULL;
    if (!aligned({u, delta, B, C, z, state, conv_state, out}, 16) ||
        !aligned({A, Dskip, delta_bias, slots, conv_weight, conv_bias}, 4))
        return SS_ERR_ALIGN;
    if (ceil_div(D, 32) * b > kMaxI32)
        return SS_ERR_SHAPE;
    if (b * D == 0)
        return SS_OK;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if ((st = check_stream(strm)) != SS_OK)
        return st;
    so::StepParams p;
    p.u = u;
    p.delta = delta;
    p.B = B;
    p.C = C;
    p.z = z;
    p.A = A;
    p.Dskip = Dskip;
    p.bias = delta_bias;
    p.conv_w = conv_weight;
    p.conv_b = conv_bias;
    p.state = state;
    p.slots = slots;
    p.conv_state = conv_state;
    p.out = out;
    p.batch = b;
    p.D = D;
    p.num_slots = num_slots;
    p.N = static_cast<int32_t>(shape->dstate);
    p.softplus = softplus ? 1 : 0;
    p.conv_width = conv_width;
    return status_of(so::launch_step(p, shape->io_dtype, strm));
}

static ss_status state_call(bool load, int64_t rows, int64_t dim, int64_t dstate, int32_t bits,
                            const float* state_in, float* state_out, int64_t state_slots,
                            void* codes, float* scales, int64_t cache_slots, const int32_t* src,
                            const int32_t* dst, void* stream)
{
    if (rows < 0 || rows > (int64_t{1} << 24) || dim < 0 || dim > (int64_t{1} << 24) || dstate < 1)
        return SS_ERR_SHAPE;
    if (dstate > SS_MAX_DSTATE || (bits != 8 && bits != 4))
        return SS_ERR_UNSUPPORTED;
    const int64_t from = load ? cache_slots : state_slots, to = load ? state_slots : cache_slots;
    if (from < 1 || to < 1 || from > kMaxI32 || to > kMaxI32 || (!src && from < rows) ||
        (!dst && to < rows) || ceil_div(dim, 32) * rows > kMaxI32 || (dst && rows > kMostListedRows))
        return SS_ERR_SHAPE;
    if (rows * dim > 0 && ((!state_in && !state_out) || !codes || !scales))
        return SS_ERR_NULL;
    if (!aligned({state_in, state_out, codes}, 16) || !aligned({scales, src, dst}, 4))
        return SS_ERR_ALIGN;
    if (rows * dim == 0)
        return SS_OK;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    const ss_status st = check_stream(strm);
    if (st != SS_OK)
        return st;
    so::StateParams p;
    p.state_in = state_in;
    p.state_out = state_out;
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = scales;
    p.src = src;
    p.dst = dst;
    p.src_slots = from;
    p.dst_slots = to;
    p.rows = rows;
    p.D = dim;
    p.N = static_cast<int32_t>(dstate);
    p.bits = bits;
    return status_of(so::launch_state(p, load, strm));
}

ss_status selective_state_store(int64_t rows, int64_t dim, int64_t dstate, int32_t bits,
                                const float* state, int64_t state_slots,
                                const int32_t* src_slots, void* codes, float* scales,
                                int64_t cache_slots, const int32_t* dst_slots, void* stream)
{
    return state_call(false, rows, dim, dstate, bits, state, nullptr, state_slots, codes, scales,
                      cache_slots, src_slots, dst_slots, stream);
}

ss_status selective_state_load(int64_t rows, int64_t dim, int64_t dstate, int32_t bits,
                               const void* codes, const float* scales, int64_t cache_slots,
                               const int32_t* src_slots, float* state, int64_t state_slots,
                               const int32_t* dst_slots, void* stream)
{
    return state_call(true, rows, dim, dstate, bits, nullptr, state, state_slots,
                      const_cast<void*>(codes), const_cast<float*>(scales), cache_slots, src_slots,
                      dst_slots, stream);
}

}  // extern "C"
