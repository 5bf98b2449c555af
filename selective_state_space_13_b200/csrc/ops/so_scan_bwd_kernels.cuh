// Gradient of the selective scan.
//
// Two sweeps over time tiles of kBwdTile steps.  The summary sweep runs the recurrence forward and
// stores the state at the start of every tile (a checkpoint); the gradient sweep walks the tiles
// backwards, recomputes a tile's states from its checkpoint into registers and runs the reverse
// recurrence over them.  Nothing of size batch x L x D x N crosses HBM except one state in eight.
//
// A CTA of 4 warps owns 64 channels of one (direction, batch row, segment).  A thread owns 2
// channels x 4 states: 4 lanes make a channel, so the sums over states (y, sum g B, sum g A h) and
// the sums over channels (dB, dC) are both shorter than with one thread per channel, where every
// step would add 32 values over 32 lanes.  Both kinds go through shared memory: a lane stores its
// partial sums once, and the threads that finish a (step, channel) or a (step, state) add them up.
//
// Sequences are cut into S segments when there are too few CTAs.  The summary sweep then starts
// every segment from zero and also returns, per channel and state, the product P of its decays
// and what the segment passes back in the reverse recurrence, G = sum_t (prod_{s<=t} Abar_s) C_t dy_t
// -- both need only the decays that the forward recurrence has computed anyway.  The gradient
// sweep folds those of the segments before (states) and after (gradients) its own, and adds
// exp(A sum Delta) h_start to each checkpoint.
//
// dB, dC and the parameter gradients leave each CTA as fp32 partial sums that a last launch adds
// in a fixed order.
#pragma once

#include <type_traits>

#include "so_device.cuh"

namespace so {

namespace {

constexpr int kT = kBwdTile;
constexpr int kC = kBwdChannels;
constexpr int kBwdThreads = 128;
constexpr int kNP = 16;  // states, padded

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared, zeros where !valid.
__device__ __forceinline__ void cp16(void* dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Position visited at step t (the index map of the scan orders).
__device__ __forceinline__ int64_t pos_of(int dir, int64_t L, int32_t H, int32_t W, int64_t t)
{
    if (dir == SS_DIR_FWD)
        return t;
    if (dir == SS_DIR_REV)
        return L - 1 - t;
    const uint32_t s = static_cast<uint32_t>(dir == SS_DIR_COL_REV ? L - 1 - t : t);
    const uint32_t col = s / static_cast<uint32_t>(H);
    return static_cast<int64_t>(s - col * H) * W + col;
}

struct Unit {
    int64_t kb, b, ub, c0, t0, t1, tile0;
    int64_t ctile, ctiles, ntiles;
    int k, seg, dir, cv;
};

__device__ __forceinline__ Unit unit_of(const BwdParams& p)
{
    Unit u;
    int64_t i = blockIdx.x;
    u.ctiles = (p.D + kC - 1) / kC;
    u.ctile = i % u.ctiles;
    i /= u.ctiles;
    u.kb = i % (p.batch * p.K);
    u.seg = static_cast<int>(i / (p.batch * p.K));
    u.k = static_cast<int>(u.kb / p.batch);
    u.b = u.kb - u.k * p.batch;
    u.ub = p.u_per_dir ? u.kb : u.b;
    u.dir = u.k == 0 ? p.dirs[0] : u.k == 1 ? p.dirs[1] : u.k == 2 ? p.dirs[2] : p.dirs[3];
    u.c0 = u.ctile * kC;
    u.cv = static_cast<int>(p.D - u.c0 < kC ? p.D - u.c0 : kC);
    u.t0 = u.seg * p.seg_len;
    u.t1 = u.t0 + p.seg_len < p.L ? u.t0 + p.seg_len : p.L;
    u.tile0 = u.t0 / kT;
    u.ntiles = (p.L + kT - 1) / kT;
    return u;
}

// One stage: the raw rows of a tile, and (gradient sweep) its checkpoint.
template <typename io_t> struct Stage {
    io_t u[kT][kC], delta[kT][kC], dout[kT][kC], z[kT][kC];
    float4 ckpt[2][kBwdThreads];
};

template <typename io_t> struct SumSmem {
    Stage<io_t> st[2];
    float4 scal[kT][kC];    // Delta, Delta u, dy
    float B[kT][kNP], C[kT][kNP];
};

template <typename io_t> struct GradSmem {
    Stage<io_t> st[2];
    float4 scal[kT][kC];
    float B[kT][kNP], C[kT][kNP];
    float part[3][kT][kC][4];               // y, sum g B, sum g A2 Abar h: one value per state group
    float dbc[kT][2][kBwdThreads / 4][kNP];  // dB, dC of every (warp, channel group)
};

// Starts the copies of time tile `tile` (steps t..t+rows-1) into a stage; returns the raw B and C
// elements this thread will convert.
template <typename io_t, bool GRAD>
__device__ __forceinline__ void issue(const BwdParams& p, const Unit& un, int64_t tile,
                                      Stage<io_t>& st, bool want_dy, io_t* bc)
{
    constexpr int E = 16 / sizeof(io_t);  // elements of a 16-byte piece
    constexpr int PR = kC / E;            // pieces of a row
    const int64_t t = tile * kT;
    const int rows = static_cast<int>(un.t1 - t < kT ? un.t1 - t : kT);
    const io_t* gu = static_cast<const io_t*>(p.u) + un.ub * p.L * p.D + un.c0;
    const io_t* gl = static_cast<const io_t*>(p.delta) + un.kb * p.L * p.D + un.c0;
    const io_t* go = static_cast<const io_t*>(p.dout) + un.b * p.L * p.D + un.c0;
    const io_t* gz = static_cast<const io_t*>(p.z);
#pragma unroll
    for (int i = 0; i < kT * PR / kBwdThreads + (kT * PR % kBwdThreads ? 1 : 0); ++i) {
        const int j = threadIdx.x + i * kBwdThreads;
        const int r = j / PR, c = (j % PR) * E;
        if (j < kT * PR) {
            const bool ok = r < rows && c < un.cv;
            const int64_t at = ok ? pos_of(un.dir, p.L, p.H, p.W, t + r) * p.D + c : 0;
            cp16(&st.u[r][c], gu + at, ok);
            cp16(&st.delta[r][c], gl + (ok ? (t + r) * p.D + c : 0), ok);
            if (want_dy) {
                cp16(&st.dout[r][c], go + at, ok);
                if (gz)
                    cp16(&st.z[r][c], gz + un.b * p.L * p.D + un.c0 + at, ok);
            }
        }
    }
    if (GRAD) {
        const float4* ck = reinterpret_cast<const float4*>(p.ckpt) +
                           ((un.kb * un.ntiles + tile) * un.ctiles + un.ctile) * 2 * kBwdThreads;
        cp16(&st.ckpt[0][threadIdx.x], ck + threadIdx.x, true);
        cp16(&st.ckpt[1][threadIdx.x], ck + kBwdThreads + threadIdx.x, true);
    }
    cp_commit();
    const int r = threadIdx.x / kNP, n = threadIdx.x % kNP;
    static_assert(kT * kNP == kBwdThreads, "one B and one C element a thread");
    const bool ok = r < rows && n < p.N;
    const int64_t at = (un.kb * p.L + t + r) * p.N + n;
    bc[0] = ok ? static_cast<const io_t*>(p.B)[at] : io_t(0.f);
    bc[1] = ok ? static_cast<const io_t*>(p.C)[at] : io_t(0.f);
}

// Per-channel parameters of the two channels whose elementwise work a thread does.
struct Par {
    float2 skip, bias;
};

__device__ __forceinline__ Par load_par(const BwdParams& p, const Unit& un)
{
    const int c = 2 * (threadIdx.x & 31);
    const int64_t d = (p.params_per_dir ? un.k * p.D : 0) + un.c0 + c;
    Par q;
    q.skip = q.bias = make_float2(0.f, 0.f);
    if (c < un.cv) {
        if (p.Dskip)
            q.skip = make_float2(p.Dskip[d], p.Dskip[d + 1]);
        if (p.bias)
            q.bias = make_float2(p.bias[d], p.bias[d + 1]);
    }
    return q;
}

template <typename io_t> __device__ __forceinline__ float2 pair_at(const io_t* row, int c)
{
    return Pair<io_t>::f(*reinterpret_cast<const typename Pair<io_t>::raw*>(row + c));
}

// Delta, Delta u and dy of the tile, two channels and every fourth step a thread; steps behind
// the segment and channels behind the row become Delta = 0 (a step that changes nothing).
template <typename io_t, typename Smem>
__device__ __forceinline__ void prepass(const BwdParams& p, const Unit& un, int64_t tile, Smem& sm,
                                        const Stage<io_t>& st, const Par& par, bool want_dy,
                                        const io_t* bc)
{
    const int c = 2 * (threadIdx.x & 31);
    const int rows = static_cast<int>(un.t1 - tile * kT < kT ? un.t1 - tile * kT : kT);
#pragma unroll
    for (int r = threadIdx.x >> 5; r < kT; r += kBwdThreads / 32) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (r < rows && c < un.cv) {
            const float2 u = pair_at(st.u[r], c), l = pair_at(st.delta[r], c);
            a.x = l.x + par.bias.x;
            b.x = l.y + par.bias.y;
            if (p.softplus) {
                a.x = softplus_f(a.x);
                b.x = softplus_f(b.x);
            }
            a.y = a.x * u.x;
            b.y = b.x * u.y;
            if (want_dy) {
                const float2 o = pair_at(st.dout[r], c);
                a.z = o.x;
                b.z = o.y;
                if (p.z) {
                    const float2 z = pair_at(st.z[r], c);
                    a.z *= silu_f(z.x);
                    b.z *= silu_f(z.y);
                }
            }
        }
        sm.scal[r][c] = a;
        sm.scal[r][c + 1] = b;
    }
    const int r = threadIdx.x / kNP, n = threadIdx.x % kNP;
    sm.B[r][n] = ld1(&bc[0]);
    sm.C[r][n] = ld1(&bc[1]);
}

// The thread's 2 channels x 4 states.
struct Cell {
    int ng, c[2];
};

__device__ __forceinline__ Cell cell_of()
{
    Cell x;
    const int lane = threadIdx.x & 31;
    x.ng = lane & 3;
    x.c[0] = (threadIdx.x >> 5) * 16 + (lane >> 2);
    x.c[1] = x.c[0] + 8;
    return x;
}

__device__ __forceinline__ void load_A2(const BwdParams& p, const Unit& un, const Cell& x,
                                        float2 A2[2][2])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * x.ng + i;
            const int64_t d = (p.params_per_dir ? un.k * p.D : 0) + un.c0 + x.c[j];
            a[i] = x.c[j] < un.cv && n < p.N ? p.A[d * p.N + n] * kLog2e : 0.f;
        }
        A2[j][0] = make_float2(a[0], a[1]);
        A2[j][1] = make_float2(a[2], a[3]);
    }
}

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// Index of this thread's states in [K*batch, S, D, 16] arrays (channel j).
__device__ __forceinline__ int64_t seg_at(const BwdParams& p, const Unit& un, const Cell& x, int seg,
                                          int j)
{
    return ((un.kb * p.S + seg) * p.D + un.c0 + x.c[j]) * kNP + 4 * x.ng;
}

// ------------------------------------------------------------------------- summary sweep

template <typename io_t, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads) summary_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw_smem[];
    SumSmem<io_t>& sm = *reinterpret_cast<SumSmem<io_t>*>(raw_smem);
    const Unit un = unit_of(p);
    const Cell x = cell_of();
    const Par par = load_par(p, un);
    float2 A2[2][2], h[2][2], P[2][2], G[2][2];
    load_A2(p, un, x, A2);
    float cum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[j][i] = G[j][i] = dup(0.f);
            P[j][i] = dup(1.f);
        }
    const int64_t ntile = (un.t1 - un.t0 + kT - 1) / kT;
    io_t bc[2];
    issue<io_t, false>(p, un, un.tile0, sm.st[0], SPLIT, bc);
    for (int64_t it = 0; it < ntile; ++it) {
        const int64_t tile = un.tile0 + it;
        cp_wait_all();
        __syncthreads();
        prepass(p, un, tile, sm, sm.st[it & 1], par, SPLIT, bc);
        __syncthreads();
        if (it + 1 < ntile)
            issue<io_t, false>(p, un, tile + 1, sm.st[(it + 1) & 1], SPLIT, bc);
        float4* ck = reinterpret_cast<float4*>(p.ckpt) +
                     ((un.kb * un.ntiles + tile) * un.ctiles + un.ctile) * 2 * kBwdThreads;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ck[j * kBwdThreads + threadIdx.x] =
                make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
            if (SPLIT && x.ng == 0 && x.c[j] < un.cv)
                p.cum[(un.kb * un.ntiles + tile) * p.D + un.c0 + x.c[j]] = cum[j];
        }
#pragma unroll
        for (int r = 0; r < kT; ++r) {
            const float4 B4 = *reinterpret_cast<const float4*>(&sm.B[r][4 * x.ng]);
            const float2 B[2] = {make_float2(B4.x, B4.y), make_float2(B4.z, B4.w)};
            const float4 C4 = *reinterpret_cast<const float4*>(&sm.C[r][4 * x.ng]);
            const float2 C[2] = {make_float2(C4.x, C4.y), make_float2(C4.z, C4.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 s = sm.scal[r][x.c[j]];
                if (SPLIT)
                    cum[j] += s.x;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 a = ex2_2(__fmul2_rn(dup(s.x), A2[j][i]));
                    h[j][i] = __ffma2_rn(a, h[j][i], __fmul2_rn(dup(s.y), B[i]));
                    if (SPLIT) {
                        P[j][i] = __fmul2_rn(P[j][i], a);
                        G[j][i] = __ffma2_rn(P[j][i], __fmul2_rn(dup(s.z), C[i]), G[j][i]);
                    }
                }
            }
        }
    }
    if (SPLIT) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (x.c[j] < un.cv) {
                const int64_t at = seg_at(p, un, x, un.seg, j);
                *reinterpret_cast<float4*>(p.seg_h + at) =
                    make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
                *reinterpret_cast<float4*>(p.seg_p + at) =
                    make_float4(P[j][0].x, P[j][0].y, P[j][1].x, P[j][1].y);
                *reinterpret_cast<float4*>(p.seg_g + at) =
                    make_float4(G[j][0].x, G[j][0].y, G[j][1].x, G[j][1].y);
            }
    }
}

// ------------------------------------------------------------------------- gradient sweep

// The elementwise end of a tile, two channels and every fourth step a thread, and the sums of its
// dB and dC over the CTA's channels.
template <typename io_t>
__device__ __forceinline__ void finish_tile(const BwdParams& p, const Unit& un, int64_t tile,
                                            GradSmem<io_t>& sm, const Stage<io_t>& st, const Par& par,
                                            float2& dskip, float2& dbias)
{
    using P2 = Pair<io_t>;
    using raw = typename P2::raw;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = 2 * lane;
    const int64_t t = tile * kT;
    const int rows = static_cast<int>(un.t1 - t < kT ? un.t1 - t : kT);
#pragma unroll
    for (int r = warp; r < kT; r += kBwdThreads / 32)
        if (r < rows && c < un.cv) {
            float du[2], dl[2], dz[2];
            const float2 u2 = pair_at(st.u[r], c), l2 = pair_at(st.delta[r], c);
            const float2 o2 = pair_at(st.dout[r], c);
            const float2 z2 = p.z ? pair_at(st.z[r], c) : make_float2(0.f, 0.f);
            const float u[2] = {u2.x, u2.y}, o[2] = {o2.x, o2.y}, z[2] = {z2.x, z2.y};
            const float l[2] = {l2.x + par.bias.x, l2.y + par.bias.y};
            const float skip[2] = {par.skip.x, par.skip.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 s = sm.scal[r][c + j];
                const float4 b4 = *reinterpret_cast<const float4*>(sm.part[1][r][c + j]);
                const float4 a4 = *reinterpret_cast<const float4*>(sm.part[2][r][c + j]);
                const float gB = (b4.x + b4.y) + (b4.z + b4.w);
                const float gA = ((a4.x + a4.y) + (a4.z + a4.w)) * kLn2;
                du[j] = fmaf(skip[j], s.z, s.x * gB);
                dl[j] = fmaf(u[j], gB, gA);
                if (p.softplus)
                    dl[j] *= sigmoid_f(l[j]);
                if (p.z) {
                    const float4 y4 = *reinterpret_cast<const float4*>(sm.part[0][r][c + j]);
                    const float y = fmaf(skip[j], u[j], (y4.x + y4.y) + (y4.z + y4.w));
                    const float sg = sigmoid_f(z[j]);
                    dz[j] = o[j] * y * sg * fmaf(z[j], 1.f - sg, 1.f);
                }
            }
            const float4 s0 = sm.scal[r][c], s1 = sm.scal[r][c + 1];
            dskip.x = fmaf(s0.z, u[0], dskip.x);
            dskip.y = fmaf(s1.z, u[1], dskip.y);
            dbias.x += dl[0];
            dbias.y += dl[1];
            const int64_t at = pos_of(un.dir, p.L, p.H, p.W, t + r) * p.D + un.c0 + c;
            if (p.du_part)
                *reinterpret_cast<float2*>(p.du_part + un.kb * p.L * p.D + at) =
                    make_float2(du[0], du[1]);
            else
                *reinterpret_cast<raw*>(static_cast<io_t*>(p.g.du) + un.ub * p.L * p.D + at) =
                    P2::r(make_float2(du[0], du[1]));
            *reinterpret_cast<raw*>(static_cast<io_t*>(p.g.ddelta) + (un.kb * p.L + t + r) * p.D +
                                    un.c0 + c) = P2::r(make_float2(dl[0], dl[1]));
            if (p.z) {
                if (p.dz_part)
                    *reinterpret_cast<float2*>(p.dz_part + un.kb * p.L * p.D + at) =
                        make_float2(dz[0], dz[1]);
                else
                    *reinterpret_cast<raw*>(static_cast<io_t*>(p.g.dz) + un.b * p.L * p.D + at) =
                        P2::r(make_float2(dz[0], dz[1]));
            }
        }
    // dB and dC: a pair of threads adds the 32 partial rows of one (step, tensor, 4 states)
    const int half = (lane >> 2) & 1, n4 = 4 * (lane & 3);
    const int which = warp * 4 + (lane >> 3);
    const int r = which >> 1, q = which & 1;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kBwdThreads / 8; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(&sm.dbc[r][q][2 * i + half][n4]);
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
    }
    v.x += __shfl_xor_sync(0xffffffffu, v.x, 4);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, 4);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, 4);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, 4);
    if (half == 0 && r < rows)
        *reinterpret_cast<float4*>(p.dbc + ((un.kb * un.ctiles + un.ctile) * p.L + t + r) * 2 * kNP +
                                   q * kNP + n4) = v;
}

template <typename io_t, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads) grad_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw_smem[];
    GradSmem<io_t>& sm = *reinterpret_cast<GradSmem<io_t>*>(raw_smem);
    const Unit un = unit_of(p);
    const Cell x = cell_of();
    const Par par = load_par(p, un);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 A2[2][2], g[2][2], dA[2][2], hstart[2][2];
    load_A2(p, un, x, A2);
    float2 dskip = dup(0.f), dbias = dup(0.f);

    // the state that enters the segment and the gradient that enters it from behind
    const bool shift = SPLIT && (un.seg > 0 || p.init != nullptr);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float hv[4], gv[4];
        const int64_t at = (un.kb * p.D + un.c0 + x.c[j]) * p.N + 4 * x.ng;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool ok = x.c[j] < un.cv && 4 * x.ng + i < p.N;
            hv[i] = ok && p.init ? p.init[at + i] : 0.f;
            gv[i] = ok && p.dlast ? p.dlast[at + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            hstart[j][i] = make_float2(hv[2 * i], hv[2 * i + 1]);
            g[j][i] = make_float2(gv[2 * i], gv[2 * i + 1]);
            dA[j][i] = dup(0.f);
        }
        if (SPLIT && x.c[j] < un.cv) {
            for (int s = 0; s < un.seg; ++s) {
                const int64_t o = seg_at(p, un, x, s, j);
                const float4 P = *reinterpret_cast<const float4*>(p.seg_p + o);
                const float4 H = *reinterpret_cast<const float4*>(p.seg_h + o);
                hstart[j][0] = __ffma2_rn(make_float2(P.x, P.y), hstart[j][0], make_float2(H.x, H.y));
                hstart[j][1] = __ffma2_rn(make_float2(P.z, P.w), hstart[j][1], make_float2(H.z, H.w));
            }
            for (int s = p.S - 1; s > un.seg; --s) {
                const int64_t o = seg_at(p, un, x, s, j);
                const float4 P = *reinterpret_cast<const float4*>(p.seg_p + o);
                const float4 G = *reinterpret_cast<const float4*>(p.seg_g + o);
                g[j][0] = __ffma2_rn(make_float2(P.x, P.y), g[j][0], make_float2(G.x, G.y));
                g[j][1] = __ffma2_rn(make_float2(P.z, P.w), g[j][1], make_float2(G.z, G.w));
            }
        }
    }

    const int64_t ntile = (un.t1 - un.t0 + kT - 1) / kT;
    io_t bc[2];
    issue<io_t, true>(p, un, un.tile0 + ntile - 1, sm.st[(ntile - 1) & 1], true, bc);
    for (int64_t it = ntile - 1; it >= 0; --it) {
        const int64_t tile = un.tile0 + it;
        const Stage<io_t>& st = sm.st[it & 1];
        cp_wait_all();
        __syncthreads();
        // the sums of the tile done before this one, while its rows are still in their stage
        if (it + 1 < ntile) {
            finish_tile(p, un, tile + 1, sm, sm.st[(it + 1) & 1], par, dskip, dbias);
            __syncthreads();  // scal is rewritten below
        }
        prepass(p, un, tile, sm, st, par, true, bc);
        __syncthreads();
        if (it > 0)
            issue<io_t, true>(p, un, tile - 1, sm.st[(it - 1) & 1], true, bc);

        // the tile's states, from its checkpoint
        float2 h[kT + 1][2][2], a[kT][2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 ck = st.ckpt[j][threadIdx.x];
            h[0][j][0] = make_float2(ck.x, ck.y);
            h[0][j][1] = make_float2(ck.z, ck.w);
            if (shift) {
                const float cum = x.c[j] < un.cv
                                      ? p.cum[(un.kb * un.ntiles + tile) * p.D + un.c0 + x.c[j]]
                                      : 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    h[0][j][i] = __ffma2_rn(ex2_2(__fmul2_rn(dup(cum), A2[j][i])), hstart[j][i],
                                            h[0][j][i]);
            }
        }
#pragma unroll
        for (int r = 0; r < kT; ++r) {
            const float4 B4 = *reinterpret_cast<const float4*>(&sm.B[r][4 * x.ng]);
            const float2 B[2] = {make_float2(B4.x, B4.y), make_float2(B4.z, B4.w)};
            const float4 C4 = *reinterpret_cast<const float4*>(&sm.C[r][4 * x.ng]);
            const float2 C[2] = {make_float2(C4.x, C4.y), make_float2(C4.z, C4.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 s = sm.scal[r][x.c[j]];
                float2 y = dup(0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[r][j][i] = ex2_2(__fmul2_rn(dup(s.x), A2[j][i]));
                    h[r + 1][j][i] = __ffma2_rn(a[r][j][i], h[r][j][i], __fmul2_rn(dup(s.y), B[i]));
                    y = __ffma2_rn(C[i], h[r + 1][j][i], y);
                }
                if (p.z)
                    sm.part[0][r][x.c[j]][x.ng] = y.x + y.y;
            }
        }
        // the reverse recurrence
#pragma unroll
        for (int r = kT - 1; r >= 0; --r) {
            const float4 B4 = *reinterpret_cast<const float4*>(&sm.B[r][4 * x.ng]);
            const float2 B[2] = {make_float2(B4.x, B4.y), make_float2(B4.z, B4.w)};
            const float4 C4 = *reinterpret_cast<const float4*>(&sm.C[r][4 * x.ng]);
            const float2 C[2] = {make_float2(C4.x, C4.y), make_float2(C4.z, C4.w)};
            float2 dB[2] = {dup(0.f), dup(0.f)}, dC[2] = {dup(0.f), dup(0.f)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 s = sm.scal[r][x.c[j]];
                float2 gB = dup(0.f), gA = dup(0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    g[j][i] = __ffma2_rn(dup(s.z), C[i], g[j][i]);
                    dC[i] = __ffma2_rn(dup(s.z), h[r + 1][j][i], dC[i]);
                    dB[i] = __ffma2_rn(dup(s.y), g[j][i], dB[i]);
                    gB = __ffma2_rn(g[j][i], B[i], gB);
                    g[j][i] = __fmul2_rn(g[j][i], a[r][j][i]);
                    const float2 q = __fmul2_rn(g[j][i], h[r][j][i]);
                    gA = __ffma2_rn(q, A2[j][i], gA);
                    dA[j][i] = __ffma2_rn(q, dup(s.x), dA[j][i]);
                }
                sm.part[1][r][x.c[j]][x.ng] = gB.x + gB.y;
                sm.part[2][r][x.c[j]][x.ng] = gA.x + gA.y;
            }
            const int row = warp * 8 + (lane >> 2);
            *reinterpret_cast<float4*>(&sm.dbc[r][0][row][4 * x.ng]) =
                make_float4(dB[0].x, dB[0].y, dB[1].x, dB[1].y);
            *reinterpret_cast<float4*>(&sm.dbc[r][1][row][4 * x.ng]) =
                make_float4(dC[0].x, dC[0].y, dC[1].x, dC[1].y);
        }
    }
    __syncthreads();
    finish_tile(p, un, un.tile0, sm, sm.st[0], par, dskip, dbias);

    // what the segment leaves: the initial state's gradient and its parameter gradients
    const int64_t row = un.kb * p.S + un.seg;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * x.ng + i;
            if (x.c[j] < un.cv && n < p.N) {
                const float2 gv = g[j][i / 2], av = dA[j][i / 2];
                const int64_t d = un.c0 + x.c[j];
                if (p.g.dinitial_state && un.seg == 0)
                    p.g.dinitial_state[(un.kb * p.D + d) * p.N + n] = i & 1 ? gv.y : gv.x;
                p.dpar[(row * p.D + d) * (kNP + 2) + n] = i & 1 ? av.y : av.x;
            }
        }
    __syncthreads();  // part is free again
    float* red = &sm.part[0][0][0][0];
    const int c = 2 * lane;
    red[warp * kC + c] = dskip.x;
    red[warp * kC + c + 1] = dskip.y;
    red[(4 + warp) * kC + c] = dbias.x;
    red[(4 + warp) * kC + c + 1] = dbias.y;
    __syncthreads();
    const int cc = threadIdx.x & (kC - 1), q = threadIdx.x / kC;
    if (cc < un.cv) {
        const float* r4 = red + 4 * q * kC + cc;
        p.dpar[(row * p.D + un.c0 + cc) * (kNP + 2) + kNP + q] =
            (r4[0] + r4[kC]) + (r4[2 * kC] + r4[3 * kC]);
    }
}

// ------------------------------------------------------------------------- the last sums

// dB, dC = sum over the channel tiles; a thread has one element.
template <typename io_t>
__global__ void __launch_bounds__(256) sum_dbc_kernel(const __grid_constant__ BwdParams p)
{
    const int64_t i = blockIdx.x * int64_t{256} + threadIdx.x;
    const int64_t ctiles = (p.D + kC - 1) / kC;
    if (i >= p.K * p.batch * p.L * 2 * kNP)
        return;
    const int64_t row = i / (2 * kNP);  // kb * L + t
    const int j = static_cast<int>(i % (2 * kNP));
    const int64_t kb = row / p.L, t = row - kb * p.L;
    const float* src = p.dbc + (kb * ctiles * p.L + t) * 2 * kNP + j;
    float v = 0.f;
    for (int64_t c = 0; c < ctiles; ++c)
        v += src[c * p.L * 2 * kNP];
    const int n = j % kNP;
    if (n < p.N)
        st1(static_cast<io_t*>(j < kNP ? p.g.dB : p.g.dC) + row * p.N + n, v);
}

// dA, dDskip, ddelta_bias = sum over (direction,) batch rows and segments: 32 columns by 8 groups
// of rows a CTA.
__global__ void __launch_bounds__(256) sum_par_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ float s[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t cols = p.D * (kNP + 2);
    const int64_t col = blockIdx.x * int64_t{32} + x;
    const int64_t sets = p.params_per_dir ? p.K : 1;
    const int64_t rows = p.K * p.batch * p.S / sets;
    const int64_t set = blockIdx.y;
    const int64_t d = col / (kNP + 2);
    const int j = static_cast<int>(col - d * (kNP + 2));
    const bool used = col < cols && (j < p.N || j >= kNP);
    float v = 0.f;
    if (used)
        for (int64_t r = y; r < rows; r += 8)
            v += p.dpar[(set * rows + r) * cols + col];
    s[y][x] = v;
    __syncthreads();
    if (y == 0 && used) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v += s[i][x];
        if (j < p.N)
            p.g.dA[(set * p.D + d) * p.N + j] = v;
        else if (j == kNP && p.g.dDskip)
            p.g.dDskip[set * p.D + d] = v;
        else if (j == kNP + 1 && p.g.ddelta_bias)
            p.g.ddelta_bias[set * p.D + d] = v;
    }
}

// du or dz = sum over the directions' parts, four elements a thread.
template <typename io_t>
__global__ void __launch_bounds__(256) sum_dirs_kernel(const float* part, io_t* out, int64_t n, int K)
{
    using P2 = Pair<io_t>;
    const int64_t i = 4 * (blockIdx.x * int64_t{256} + threadIdx.x);
    if (i >= n)
        return;
    float4 v = *reinterpret_cast<const float4*>(part + i);
    for (int k = 1; k < K; ++k) {
        const float4 w = *reinterpret_cast<const float4*>(part + k * n + i);
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
    }
    typename P2::raw* o = reinterpret_cast<typename P2::raw*>(out + i);
    o[0] = P2::r(make_float2(v.x, v.y));
    o[1] = P2::r(make_float2(v.z, v.w));
}

template <typename io_t, bool SPLIT> cudaError_t launch_sweeps(const BwdParams& p, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(summary_kernel<io_t, SPLIT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         sizeof(SumSmem<io_t>));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grad_kernel<io_t, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 sizeof(GradSmem<io_t>));
    if (e != cudaSuccess)
        return e;
    const unsigned blocks =
        static_cast<unsigned>((p.D + kC - 1) / kC * p.batch * p.K * p.S);
    summary_kernel<io_t, SPLIT><<<blocks, kBwdThreads, sizeof(SumSmem<io_t>), st>>>(p);
    grad_kernel<io_t, SPLIT><<<blocks, kBwdThreads, sizeof(GradSmem<io_t>), st>>>(p);
    return cudaGetLastError();
}

template <typename io_t> cudaError_t launch_bwd_io(const BwdParams& p, cudaStream_t st)
{
    cudaError_t e = p.S > 1 || p.init ? launch_sweeps<io_t, true>(p, st)
                                      : launch_sweeps<io_t, false>(p, st);
    if (e != cudaSuccess)
        return e;
    const int64_t nbc = p.K * p.batch * p.L * 2 * kNP;
    sum_dbc_kernel<io_t><<<static_cast<unsigned>((nbc + 255) / 256), 256, 0, st>>>(p);
    const dim3 grid(static_cast<unsigned>((p.D * (kNP + 2) + 31) / 32), p.params_per_dir ? p.K : 1);
    sum_par_kernel<<<grid, 256, 0, st>>>(p);
    const int64_t n = p.batch * p.L * p.D;
    const unsigned nb = static_cast<unsigned>((n / 4 + 255) / 256);
    if (p.du_part)
        sum_dirs_kernel<io_t><<<nb, 256, 0, st>>>(p.du_part, static_cast<io_t*>(p.g.du), n, p.K);
    if (p.dz_part)
        sum_dirs_kernel<io_t><<<nb, 256, 0, st>>>(p.dz_part, static_cast<io_t*>(p.g.dz), n, p.K);
    return cudaGetLastError();
}

}  // namespace

}  // namespace so
