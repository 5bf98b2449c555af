// Gated linear recurrence h_t = a_t h_{t-1} + c_t x_t and its gradient.
//
// Every channel is a chain of scalar affine maps, so a sequence cut into S segments needs only the
// pair (P, H) of each segment (product of its decays, end state from zero): a first launch
// computes the pairs of all segments but the last (the first, in the gradient), a second one folds
// the pairs before its segment and runs the segment.  One thread owns two adjacent channels.
#include "so_device.cuh"

namespace so {

namespace {

constexpr int kThreads = 64;
constexpr int kCh = 2 * kThreads;  // channels of a CTA
constexpr int kUnroll = 8;         // steps whose loads are in flight together

struct Gate {
    float a, c, rest;  // decay, input factor, 1 - decay
};

template <int FORM, bool COMP> __device__ __forceinline__ Gate make_gate(float s)
{
    Gate g;
    if (FORM == SS_GATE_SIGMOID) {
        // one exponential and one reciprocal serve sigmoid(s) and sigmoid(-s)
        const float e = ex2(-fabsf(s) * kLog2e);
        const float r = rcp(1.f + e);
        const float er = e * r;
        g.a = s >= 0.f ? r : er;
        g.rest = s >= 0.f ? er : r;
    } else {
        g.a = ex2(s * kLog2e);
        g.rest = COMP ? one_minus_exp(s, g.a) : 0.f;
    }
    g.c = COMP ? g.rest : 1.f;
    return g;
}

struct Where {
    int64_t b, seg, d, t0, t1;
    bool active;
};

__device__ __forceinline__ Where where(const RecParams& p, int nseg, int seg0)
{
    Where w;
    const int64_t tiles = (p.D + kCh - 1) / kCh;
    int64_t i = blockIdx.x;
    w.d = (i % tiles) * kCh + 2 * threadIdx.x;
    i /= tiles;
    w.seg = i % nseg + seg0;
    w.b = i / nseg;
    w.t0 = w.seg * p.seg_len;
    w.t1 = w.t0 + p.seg_len < p.L ? w.t0 + p.seg_len : p.L;
    w.active = w.d < p.D;
    return w;
}

// Element offset of step t of row block b.
__device__ __forceinline__ int64_t at(const RecParams& p, int64_t b, int64_t t, int64_t d)
{
    return (b * p.L + (p.reverse ? p.L - 1 - t : t)) * p.D + d;
}

template <typename io_t, int FORM, bool COMP, bool AGG>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const RecParams p)
{
    using P2 = Pair<io_t>;
    using raw = typename P2::raw;
    const Where w = where(p, AGG ? p.S - 1 : p.S, 0);
    if (!w.active)
        return;
    const io_t* gx = static_cast<const io_t*>(p.x);
    const io_t* gg = static_cast<const io_t*>(p.gate);
    const float2 bias = p.bias ? make_float2(p.bias[w.d], p.bias[w.d + 1]) : make_float2(0.f, 0.f);
    float2 h = make_float2(0.f, 0.f), prod = make_float2(1.f, 1.f);
    if (!AGG) {
        if (p.init)
            h = make_float2(p.init[w.b * p.D + w.d], p.init[w.b * p.D + w.d + 1]);
        for (int64_t s = 0; s < w.seg; ++s) {
            const float4 c = *reinterpret_cast<const float4*>(p.carry + (w.b * p.S + s) * p.D + w.d);
            h.x = fmaf(c.x, h.x, c.y);
            h.y = fmaf(c.z, h.y, c.w);
        }
    }
    for (int64_t t = w.t0; t < w.t1; t += kUnroll) {
        raw rx[kUnroll], rg[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (t + i < w.t1) {
                const int64_t o = at(p, w.b, t + i, w.d);
                rx[i] = *reinterpret_cast<const raw*>(gx + o);
                rg[i] = *reinterpret_cast<const raw*>(gg + o);
            }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (t + i < w.t1) {
                const float2 x = P2::f(rx[i]), g = P2::f(rg[i]);
                const Gate g0 = make_gate<FORM, COMP>(g.x + bias.x);
                const Gate g1 = make_gate<FORM, COMP>(g.y + bias.y);
                h.x = fmaf(g0.a, h.x, g0.c * x.x);
                h.y = fmaf(g1.a, h.y, g1.c * x.y);
                if (AGG) {
                    prod.x *= g0.a;
                    prod.y *= g1.a;
                } else {
                    *reinterpret_cast<raw*>(static_cast<io_t*>(p.out) + at(p, w.b, t + i, w.d)) =
                        P2::r(h);
                }
            }
    }
    if (AGG) {
        *reinterpret_cast<float4*>(p.carry + (w.b * p.S + w.seg) * p.D + w.d) =
            make_float4(prod.x, h.x, prod.y, h.y);
    } else if (p.last && w.seg == p.S - 1) {
        p.last[w.b * p.D + w.d] = h.x;
        p.last[w.b * p.D + w.d + 1] = h.y;
    }
}

template <typename io_t, int FORM, bool COMP, bool AGG>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const RecParams p)
{
    using P2 = Pair<io_t>;
    using raw = typename P2::raw;
    const Where w = where(p, AGG ? p.S - 1 : p.S, AGG ? 1 : 0);
    if (!w.active)
        return;
    const io_t* gx = static_cast<const io_t*>(p.x);
    const io_t* gg = static_cast<const io_t*>(p.gate);
    const io_t* gh = static_cast<const io_t*>(p.out_in);
    const io_t* gd = static_cast<const io_t*>(p.dout);
    const float2 bias = p.bias ? make_float2(p.bias[w.d], p.bias[w.d + 1]) : make_float2(0.f, 0.f);
    float2 q = make_float2(0.f, 0.f), prod = make_float2(1.f, 1.f), db = make_float2(0.f, 0.f);
    if (!AGG) {
        if (p.dlast)
            q = make_float2(p.dlast[w.b * p.D + w.d], p.dlast[w.b * p.D + w.d + 1]);
        for (int64_t s = p.S - 1; s > w.seg; --s) {
            const float4 c = *reinterpret_cast<const float4*>(p.carry + (w.b * p.S + s) * p.D + w.d);
            q.x = fmaf(c.x, q.x, c.y);
            q.y = fmaf(c.z, q.y, c.w);
        }
    }
    for (int64_t t = w.t1; t > w.t0; t -= kUnroll) {
        raw rx[kUnroll], rg[kUnroll], rh[kUnroll], rd[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t tt = t - 1 - i;
            if (tt >= w.t0) {
                const int64_t o = at(p, w.b, tt, w.d);
                rg[i] = *reinterpret_cast<const raw*>(gg + o);
                rd[i] = *reinterpret_cast<const raw*>(gd + o);
                if (!AGG) {
                    if (COMP)
                        rx[i] = *reinterpret_cast<const raw*>(gx + o);
                    if (tt > 0)
                        rh[i] = *reinterpret_cast<const raw*>(gh + at(p, w.b, tt - 1, w.d));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t tt = t - 1 - i;
            if (tt >= w.t0) {
                const float2 g = P2::f(rg[i]), dy = P2::f(rd[i]);
                const Gate g0 = make_gate<FORM, COMP>(g.x + bias.x);
                const Gate g1 = make_gate<FORM, COMP>(g.y + bias.y);
                const float2 G = make_float2(dy.x + q.x, dy.y + q.y);
                q = make_float2(g0.a * G.x, g1.a * G.y);
                if (AGG) {
                    prod.x *= g0.a;
                    prod.y *= g1.a;
                } else {
                    float2 before = make_float2(0.f, 0.f);
                    if (tt > 0)
                        before = P2::f(rh[i]);
                    else if (p.init)
                        before = make_float2(p.init[w.b * p.D + w.d], p.init[w.b * p.D + w.d + 1]);
                    if (COMP) {
                        const float2 x = P2::f(rx[i]);
                        before.x -= x.x;
                        before.y -= x.y;
                    }
                    float2 ds = make_float2(q.x * before.x, q.y * before.y);
                    if (FORM == SS_GATE_SIGMOID) {
                        ds.x *= g0.rest;
                        ds.y *= g1.rest;
                    }
                    db.x += ds.x;
                    db.y += ds.y;
                    const int64_t o = at(p, w.b, tt, w.d);
                    *reinterpret_cast<raw*>(static_cast<io_t*>(p.out) + o) =
                        P2::r(make_float2(g0.c * G.x, g1.c * G.y));
                    *reinterpret_cast<raw*>(static_cast<io_t*>(p.dgate) + o) = P2::r(ds);
                }
            }
        }
    }
    if (AGG) {
        *reinterpret_cast<float4*>(p.carry + (w.b * p.S + w.seg) * p.D + w.d) =
            make_float4(prod.x, q.x, prod.y, q.y);
        return;
    }
    if (p.last && w.seg == 0) {
        p.last[w.b * p.D + w.d] = q.x;
        p.last[w.b * p.D + w.d + 1] = q.y;
    }
    if (p.dbias_part)
        *reinterpret_cast<float2*>(p.dbias_part + (w.b * p.S + w.seg) * p.D + w.d) = db;
}

// out[d] = sum over rows of part[row, d], in a fixed order: 32 channels by 8 row groups a CTA.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float* part, float* out, int64_t rows,
                                                       int64_t D)
{
    __shared__ float s[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t d = blockIdx.x * int64_t{32} + x;
    float v = 0.f;
    if (d < D)
        for (int64_t r = y; r < rows; r += 8)
            v += part[r * D + d];
    s[y][x] = v;
    __syncthreads();
    if (y == 0 && d < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v += s[i][x];
        out[d] = v;
    }
}

template <typename io_t, int FORM, bool COMP>
cudaError_t launch(const RecParams& p, bool backward, cudaStream_t st)
{
    const int64_t tiles = (p.D + kCh - 1) / kCh;
    const unsigned all = static_cast<unsigned>(tiles * p.batch * p.S);
    const unsigned agg = static_cast<unsigned>(tiles * p.batch * (p.S - 1));
    if (!backward) {
        if (agg)
            fwd_kernel<io_t, FORM, COMP, true><<<agg, kThreads, 0, st>>>(p);
        fwd_kernel<io_t, FORM, COMP, false><<<all, kThreads, 0, st>>>(p);
    } else {
        if (agg)
            bwd_kernel<io_t, FORM, COMP, true><<<agg, kThreads, 0, st>>>(p);
        bwd_kernel<io_t, FORM, COMP, false><<<all, kThreads, 0, st>>>(p);
        if (p.dbias)
            sum_rows_kernel<<<static_cast<unsigned>((p.D + 31) / 32), 256, 0, st>>>(
                p.dbias_part, p.dbias, p.batch * p.S, p.D);
    }
    return cudaGetLastError();
}

template <typename io_t>
cudaError_t launch_io(const RecParams& p, bool backward, cudaStream_t st)
{
    if (p.form == SS_GATE_SIGMOID)
        return p.complement ? launch<io_t, SS_GATE_SIGMOID, true>(p, backward, st)
                            : launch<io_t, SS_GATE_SIGMOID, false>(p, backward, st);
    return p.complement ? launch<io_t, SS_GATE_EXP, true>(p, backward, st)
                        : launch<io_t, SS_GATE_EXP, false>(p, backward, st);
}

}  // namespace

cudaError_t launch_recurrence(const RecParams& p, int io_dtype, bool backward, cudaStream_t st)
{
    return io_dtype == SS_BF16 ? launch_io<__nv_bfloat16>(p, backward, st)
                               : launch_io<float>(p, backward, st);
}

}  // namespace so
