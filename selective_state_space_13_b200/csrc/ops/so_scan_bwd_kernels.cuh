// Gradient of the selective scan.
//
// Two sweeps over the sequence. The summary sweep runs the recurrence forward and stores the state
// at the start of every slice of kT steps (a checkpoint); the gradient sweep walks the slices
// backwards, recomputes a slice's states from its checkpoint into registers and runs the reverse
// recurrence over them.  Nothing of size batch x L x D x N crosses HBM except one state in kT.
//
// A CTA of 4 warps owns 64 channels of one (direction, batch row, segment), a warp 16 of them, a
// thread 2 adjacent channels x 4 states: 4 lanes make a channel (for N up to 8: 128, 32, and 2 lanes;
// SO_STATE_GROUPS says which, one translation unit each).  The two channels are the halves
// of every packed f32x2 operation, so Delta, Delta u and dy come out of shared memory as pairs; B and C
// are scalars there, which a packed operation takes for both halves without moves.  The sums over
// states (y, sum g B, sum g A h) and over channels (dB, dC) go through shared memory that is private to
// the warp: a lane stores its partial sums once, and the lane that finishes a (step, channel pair) or a
// (step, 4 states) adds them up, which costs fewer instructions than a full butterfly of shuffles (one
// that halves what it keeps at every stage is not tried).
// Warps meet twice per tile of kTL steps: when its rows have landed and B and C are converted.
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
//
// A decay near one, rounded to fp32, and the error of its exponential lose up to 2^-22 of the state every
// step, which a long memory multiplies.  fp32 io gets that back once a slice: the product of the slice's
// decays, as they are, against exp(A sum Delta) - 1, which is relatively accurate (Slice).
#pragma once

#include <type_traits>

#include "so_device.cuh"
#include "ss_device.cuh"

namespace so {

namespace {

constexpr int kG = SO_STATE_GROUPS;    // groups of 4 states: 4 (N up to 16) or 2 (N up to 8)
constexpr int kNP = 4 * kG;            // states, padded
constexpr int kT = kBwdTile;           // steps of a slice
constexpr int kTL = 2 * kT;            // steps of a tile: what is loaded and prepared together
constexpr int kWarps = 4;
constexpr int kBwdThreads = 32 * kWarps;
constexpr int kWC = 64 / kG;           // channels of a warp
constexpr int kC = kWC * kWarps;       // channels of a CTA
// pitches of raw rows and of the partial sums of a step: what a warp reads together lies in
// different banks
constexpr int kPitch = kC + 64 / kG;
constexpr int kPartPitch = kG * kWC + 32 / kG;
static_assert((kG == 2 || kG == 4) && kT == 4, "lane = kG * (channel pair) + state group");
static_assert(kC == kBwdCells / kNP, "the host's plan counts the same channels");

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

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// What a CTA works on.  Element offsets inside one sequence fit in 32 bits (L * D < 2^31).
struct Unit {
    int64_t kb, b, ub;           // row blocks of delta/B/C, of dout/z, of u
    int c0, cv, ctile, ctiles;   // first channel, valid channels, channel tile
    int t0, t1, L, D;            // steps of the segment
    int k, seg, dir, H, W;

    // Element offset of the row that step t visits.
    __device__ __forceinline__ uint32_t row(int t) const
    {
        uint32_t pos = static_cast<uint32_t>(dir == SS_DIR_REV || dir == SS_DIR_COL_REV ? L - 1 - t : t);
        if (dir == SS_DIR_COL || dir == SS_DIR_COL_REV) {
            const uint32_t col = pos / static_cast<uint32_t>(H);
            pos = (pos - col * H) * W + col;
        }
        return pos * static_cast<uint32_t>(D);
    }
};

__device__ __forceinline__ Unit unit_of(const BwdParams& p)
{
    Unit u;
    u.D = static_cast<int>(p.D);
    u.L = static_cast<int>(p.L);
    u.ctiles = (u.D + kC - 1) / kC;
    unsigned i = blockIdx.x;
    u.ctile = i % u.ctiles;
    i /= u.ctiles;
    const unsigned rows = static_cast<unsigned>(p.batch * p.K);
    u.seg = i / rows;
    const unsigned kb = i % rows;
    u.k = kb / static_cast<unsigned>(p.batch);
    u.kb = kb;
    u.b = u.kb - u.k * p.batch;
    u.ub = p.u_per_dir ? u.kb : u.b;
    u.dir = u.k == 0 ? p.dirs[0] : u.k == 1 ? p.dirs[1] : u.k == 2 ? p.dirs[2] : p.dirs[3];
    u.H = p.H;
    u.W = p.W;
    u.c0 = u.ctile * kC;
    u.cv = min(u.D - u.c0, kC);
    u.t0 = static_cast<int>(u.seg * p.seg_len);
    u.t1 = static_cast<int>(min(p.L, u.seg * p.seg_len + p.seg_len));
    return u;
}

template <typename io_t> struct Stage {
    io_t u[kTL][kPitch], delta[kTL][kPitch], dout[kTL][kPitch], z[kTL][kPitch];
};

// What a CTA needs now and then: kept in shared memory and read there each time (volatile), so that
// it takes no registers from the recurrences.
struct Cta {
    const void *u, *delta, *dout, *z;  // first element of the CTA's rows and channels
    void *du, *ddelta, *dz;            // (du, dz: io rows or fp32 parts)
    const void *B, *C;
    float* dbc;
    float4* ckpt;
    float* cum;
    float skip[kC], bias[kC];
};

template <typename T> __device__ __forceinline__ T again(const T& v)
{
    return *const_cast<const volatile T*>(&v);
}

__device__ __forceinline__ float2 again2(const float* v)
{
    return make_float2(again(v[0]), again(v[1]));
}

template <typename io_t> struct SumSmem {
    Cta cta;
    Stage<io_t> st[2];
    float B[kTL][kNP], C[kTL][kNP];
    float2 scal[kWarps][kTL][3][kWC / 2];  // Delta, Delta u, dy of a channel pair
};

template <typename io_t> struct GradSmem {
    Cta cta;
    Stage<io_t> st[2];
    float B[kTL][kNP], C[kTL][kNP];
    float2 scal[kWarps][kTL][3][kWC / 2];
    float part[kWarps][3][kT][kPartPitch];  // y, sum g B, sum g A Abar h: [state group][channel]
    float dbc[kWarps][kT][2][kWC / 2][kNP]; // dB, dC of every channel pair
    float4 acc[kTL][2][kWarps][kNP / 4];    // dB, dC of every warp
    float4 hstart[2][kBwdThreads];          // the state that enters the segment (SPLIT)
};

// The CTA's bases and parameters, written once.
template <typename io_t>
__device__ __forceinline__ void fill_cta(const BwdParams& p, const Unit& un, Cta& c)
{
    const int64_t LD = p.L * p.D, nslices = (p.L + kT - 1) / kT;
    if (threadIdx.x == 0) {
        c.u = static_cast<const io_t*>(p.u) + un.ub * LD + un.c0;
        c.delta = static_cast<const io_t*>(p.delta) + un.kb * LD + un.c0;
        c.dout = static_cast<const io_t*>(p.dout) + un.b * LD + un.c0;
        c.z = static_cast<const io_t*>(p.z) + (p.z ? un.b * LD + un.c0 : 0);
        c.du = p.du_part ? static_cast<void*>(p.du_part + un.kb * LD + un.c0)
                         : static_cast<io_t*>(p.g.du) + un.ub * LD + un.c0;
        c.ddelta = static_cast<io_t*>(p.g.ddelta) + un.kb * LD + un.c0;
        c.dz = p.dz_part ? static_cast<void*>(p.dz_part + un.kb * LD + un.c0)
                         : static_cast<io_t*>(p.g.dz) + (p.z ? un.b * LD + un.c0 : 0);
        c.B = static_cast<const io_t*>(p.B) + un.kb * p.L * p.N;
        c.C = static_cast<const io_t*>(p.C) + un.kb * p.L * p.N;
        c.dbc = p.dbc + (un.kb * un.ctiles + un.ctile) * p.L * (2 * kNP);
        c.ckpt = reinterpret_cast<float4*>(p.ckpt) +
                 (un.kb * nslices * un.ctiles + un.ctile) * (2 * kBwdThreads);
        c.cum = p.cum + un.kb * nslices * p.D + un.c0;
    }
    if (threadIdx.x < kC) {
        const int64_t d = (p.params_per_dir ? un.k * p.D : 0) + un.c0 + threadIdx.x;
        const bool ok = threadIdx.x < un.cv;
        c.skip[threadIdx.x] = ok && p.Dskip ? p.Dskip[d] : 0.f;
        c.bias[threadIdx.x] = ok && p.bias ? p.bias[d] : 0.f;
    }
    __syncthreads();
}

// Starts the copies of the tile of steps t..t+kTL-1 into a stage; returns the raw B and C elements
// that this thread will convert.
constexpr int kBC = (kTL * kNP + kBwdThreads - 1) / kBwdThreads;

template <typename io_t>
__device__ __forceinline__ void issue(const BwdParams& p, const Unit& un, const Cta& cta, int t,
                                      Stage<io_t>& st, bool want_dy, io_t (*bc)[2])
{
    constexpr int E = 16 / sizeof(io_t);  // elements of a 16-byte piece
    constexpr int PR = kC / E;            // pieces of a row
    const int rows = min(un.t1 - t, kTL);
    const io_t* gu = static_cast<const io_t*>(again(cta.u));
    const io_t* gl = static_cast<const io_t*>(again(cta.delta));
    const io_t* go = static_cast<const io_t*>(again(cta.dout));
    const io_t* gz = static_cast<const io_t*>(again(cta.z));
#pragma unroll
    for (int i = 0; i < (kTL * PR + kBwdThreads - 1) / kBwdThreads; ++i) {
        const int j = threadIdx.x + i * kBwdThreads;
        if (j < kTL * PR) {
            const int r = j / PR, c = (j % PR) * E;
            const bool ok = r < rows && c < un.cv;
            const uint32_t at = ok ? un.row(t + r) + c : 0;
            cp16(&st.u[r][c], gu + at, ok);
            cp16(&st.delta[r][c], gl + (ok ? static_cast<uint32_t>(t + r) * un.D + c : 0u), ok);
            if (want_dy) {
                cp16(&st.dout[r][c], go + at, ok);
                if (p.z)
                    cp16(&st.z[r][c], gz + at, ok);
            }
        }
    }
    cp_commit();
    const io_t* gB = static_cast<const io_t*>(again(cta.B));
    const io_t* gC = static_cast<const io_t*>(again(cta.C));
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
        const int j = threadIdx.x + i * kBwdThreads, r = j / kNP, n = j % kNP;
        const bool ok = j < kTL * kNP && r < rows && n < p.N;
        const int64_t at = static_cast<int64_t>(t + r) * p.N + n;
        bc[i][0] = ok ? gB[at] : io_t(0.f);
        bc[i][1] = ok ? gC[at] : io_t(0.f);
    }
}

// The thread's place: channels c, c+1 of the CTA, states 4 ng .. 4 ng + 3; in elementwise work,
// the channel pair's steps ng, ng + kG, ... of a slice.
struct Cell {
    int warp, lane, cg, ng, c;
    bool valid;  // the channels exist (they come in pairs: D is a multiple of 4)
};

__device__ __forceinline__ Cell cell_of(const Unit& un)
{
    Cell x;
    x.lane = threadIdx.x & 31;
    x.warp = threadIdx.x >> 5;
    x.cg = x.lane / kG;
    x.ng = x.lane % kG;
    x.c = x.warp * kWC + 2 * x.cg;
    x.valid = x.c < un.cv;
    return x;
}

// A of the thread's cells, times log2(e) for the exponentials in base 2.
__device__ __forceinline__ void load_A(const BwdParams& p, const Unit& un, const Cell& x, float2 A[4])
{
    const int64_t d = (p.params_per_dir ? un.k * p.D : 0) + un.c0 + x.c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = 4 * x.ng + i;
        A[i] = dup(0.f);
        if (x.valid && n < p.N)
            A[i] = make_float2(p.A[d * p.N + n], p.A[(d + 1) * p.N + n]);
        A[i] = __fmul2_rn(A[i], dup(kLog2e));
    }
}

// The decay of a step.
template <bool PRECISE> __device__ __forceinline__ float2 decay(float2 delta, float2 A)
{
    return ex2_2(PRECISE ? __fmul2_rn(delta, A) : __ffma2_rn(delta, A, dup(kDecayShift)));
}

// What the decays of a slice have lost (PRECISE).
struct Slice {
    float2 sum, size;  // of Delta, of its magnitude
    float2 Q[4];       // the product of the decays, minus one

    __device__ __forceinline__ void start()
    {
        sum = size = Q[0] = Q[1] = Q[2] = Q[3] = dup(0.f);
    }
    __device__ __forceinline__ void step(float2 delta)
    {
        sum = __fadd2_rn(sum, delta);
        size = make_float2(size.x + fabsf(delta.x), size.y + fabsf(delta.y));
    }
    __device__ __forceinline__ void decayed_by(int i, float2 a)
    {
        const float2 c = __fadd2_rn(a, dup(-1.f));
        Q[i] = __ffma2_rn(Q[i], c, __fadd2_rn(Q[i], c));
    }
    // v with it: decays that are not near one do not come to much in the few steps that they are
    // remembered.
    __device__ __forceinline__ float2 restored(int i, float2 A, float2 v) const
    {
        // 2^x - 1 = x ln 2 (1 + x ln 2 / 2 (1 + ...)), to x^8 (below 1e-9 relative for |x| <= 1/2)
        const float2 x = __fmul2_rn(sum, A), most = __fmul2_rn(size, A);
        const float2 y = __fmul2_rn(x, dup(kLn2));
        float2 e = __ffma2_rn(y, dup(1.f / 40320.f), dup(1.f / 5040.f));
        e = __ffma2_rn(e, y, dup(1.f / 720.f));
        e = __ffma2_rn(e, y, dup(1.f / 120.f));
        e = __ffma2_rn(e, y, dup(1.f / 24.f));
        e = __ffma2_rn(e, y, dup(1.f / 6.f));
        e = __ffma2_rn(e, y, dup(0.5f));
        e = __ffma2_rn(e, y, dup(1.f));
        const float2 lost = __ffma2_rn(e, y, __fmul2_rn(Q[i], dup(-1.f)));
        return __ffma2_rn(v, make_float2(fabsf(most.x) <= 0.5f ? lost.x : 0.f,
                                         fabsf(most.y) <= 0.5f ? lost.y : 0.f), v);
    }
};

template <typename io_t> __device__ __forceinline__ float2 pair_at(const io_t* p)
{
    return Pair<io_t>::f(*reinterpret_cast<const typename Pair<io_t>::raw*>(p));
}

__device__ __forceinline__ float2 sigmoid_2(float2 x)
{
    return make_float2(sigmoid_f(x.x), sigmoid_f(x.y));
}

// softplus of a pair (softplus_f, its polynomial in packed operations).
__device__ __forceinline__ float2 softplus_2(float2 x)
{
    const float2 e = ex2_2(__fmul2_rn(make_float2(-fabsf(x.x), -fabsf(x.y)), dup(kLog2e)));
    const float2 s = __fmul2_rn(e, make_float2(rcp(2.f + e.x), rcp(2.f + e.y)));
    const float2 s2 = __fmul2_rn(s, s);
    float2 q = __ffma2_rn(dup(2.f / 15.f), s2, dup(2.f / 13.f));
    q = __ffma2_rn(q, s2, dup(2.f / 11.f));
    q = __ffma2_rn(q, s2, dup(2.f / 9.f));
    q = __ffma2_rn(q, s2, dup(2.f / 7.f));
    q = __ffma2_rn(q, s2, dup(2.f / 5.f));
    q = __ffma2_rn(q, s2, dup(2.f / 3.f));
    q = __ffma2_rn(q, s2, dup(2.f));
    return __ffma2_rn(s, q, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// Delta, Delta u and dy of the tile for the warp's channels, and B and C for the CTA.  Steps behind
// the segment and channels behind the row become Delta = 0, a step that changes nothing.
template <typename io_t, typename Smem>
__device__ __forceinline__ void prepass(const BwdParams& p, const Unit& un, const Cell& x, int t,
                                        Smem& sm, const Stage<io_t>& st, bool want_dy,
                                        const io_t (*bc)[2])
{
    const int rows = min(un.t1 - t, kTL);
    const float2 bias = again2(&sm.cta.bias[x.c]);
#pragma unroll
    for (int r = x.ng; r < kTL; r += kG) {
        float2 dl = dup(0.f), w = dl, dy = dl;
        if (r < rows && x.valid) {
            dl = __fadd2_rn(pair_at(&st.delta[r][x.c]), bias);
            if (p.softplus)
                dl = softplus_2(dl);
            w = __fmul2_rn(dl, pair_at(&st.u[r][x.c]));
            if (want_dy) {
                dy = pair_at(&st.dout[r][x.c]);
                if (p.z) {
                    const float2 z = pair_at(&st.z[r][x.c]);
                    dy = __fmul2_rn(dy, __fmul2_rn(z, sigmoid_2(z)));
                }
            }
        }
        sm.scal[x.warp][r][0][x.cg] = dl;
        sm.scal[x.warp][r][1][x.cg] = w;
        if (want_dy)
            sm.scal[x.warp][r][2][x.cg] = dy;
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
        const int j = threadIdx.x + i * kBwdThreads;
        if (j < kTL * kNP) {
            sm.B[j / kNP][j % kNP] = ld1(&bc[i][0]);
            sm.C[j / kNP][j % kNP] = ld1(&bc[i][1]);
        }
    }
}

// The thread's 4 elements of a row of B or C, each for both channels.
__device__ __forceinline__ void load4(const float (*rows)[kNP], int r, int ng, float2 v[4])
{
    const float4 a = *reinterpret_cast<const float4*>(&rows[r][4 * ng]);
    v[0] = dup(a.x);
    v[1] = dup(a.y);
    v[2] = dup(a.z);
    v[3] = dup(a.w);
}

// Per-thread arrays in global memory as two float4 per cell block.
__device__ __forceinline__ void put4(float4* at, int stride, const float2 v[4])
{
    at[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    at[stride] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

__device__ __forceinline__ void get4(const float4* at, int stride, float2 v[4])
{
    const float4 a = at[0], b = at[stride];
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
}

// Checkpoint of this thread for slice `s` of the sequence, the sums of Delta there, and the block
// of a segment.
__device__ __forceinline__ float4* ckpt_at(const Unit& un, const Cta& cta, int s)
{
    return again(cta.ckpt) + static_cast<int64_t>(s) * un.ctiles * (2 * kBwdThreads) + threadIdx.x;
}

__device__ __forceinline__ float2* cum_at(const Unit& un, const Cta& cta, const Cell& x, int s)
{
    return reinterpret_cast<float2*>(again(cta.cum) + static_cast<int64_t>(s) * un.D + x.c);
}

__device__ __forceinline__ float4* seg_at(float* base, const BwdParams& p, const Unit& un, int seg)
{
    return reinterpret_cast<float4*>(base) +
           ((un.kb * p.S + seg) * un.ctiles + un.ctile) * (2 * kBwdThreads) + threadIdx.x;
}

// ------------------------------------------------------------------------- summary sweep

template <typename io_t, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads) summary_kernel(const __grid_constant__ BwdParams p)
{
    constexpr bool PRECISE = std::is_same<io_t, float>::value;
    extern __shared__ __align__(128) unsigned char raw_smem[];
    SumSmem<io_t>& sm = *reinterpret_cast<SumSmem<io_t>*>(raw_smem);
    const Unit un = unit_of(p);
    const Cell x = cell_of(un);
    fill_cta<io_t>(p, un, sm.cta);
    float2 A[4], h[4], P[4], G[4], cum = dup(0.f);
    load_A(p, un, x, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = G[i] = dup(0.f);
        P[i] = dup(1.f);
    }
    Slice slice;
    io_t bc[kBC][2];
    issue<io_t>(p, un, sm.cta, un.t0, sm.st[0], SPLIT, bc);
    for (int t = un.t0, it = 0; t < un.t1; t += kTL, ++it) {
        cp_wait_all();
        __syncthreads();
        prepass(p, un, x, t, sm, sm.st[it & 1], SPLIT, bc);
        __syncthreads();
        if (t + kTL < un.t1)
            issue<io_t>(p, un, sm.cta, t + kTL, sm.st[(it + 1) & 1], SPLIT, bc);
#pragma unroll
        for (int r = 0; r < kTL; ++r) {
            if (r % kT == 0 && t + r < un.t1) {
                put4(ckpt_at(un, sm.cta, (t + r) / kT), kBwdThreads, h);
                if (SPLIT && x.ng == 0 && x.valid)
                    *cum_at(un, sm.cta, x, (t + r) / kT) = cum;
            }
            float2 B[4], C[4];
            load4(sm.B, r, x.ng, B);
            const float2 dl = sm.scal[x.warp][r][0][x.cg], w = sm.scal[x.warp][r][1][x.cg];
            float2 dy = dup(0.f);
            if (PRECISE) {
                if (r % kT == 0)
                    slice.start();
                slice.step(dl);
            }
            if (SPLIT) {
                load4(sm.C, r, x.ng, C);
                dy = sm.scal[x.warp][r][2][x.cg];
                cum = __fadd2_rn(cum, dl);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = decay<PRECISE>(dl, A[i]);
                h[i] = __ffma2_rn(a, h[i], __fmul2_rn(w, B[i]));
                if (SPLIT) {
                    P[i] = __fmul2_rn(a, P[i]);
                    G[i] = __ffma2_rn(P[i], __fmul2_rn(dy, C[i]), G[i]);
                }
                if (PRECISE) {
                    slice.decayed_by(i, a);
                    if (r % kT == kT - 1) {
                        h[i] = slice.restored(i, A[i], h[i]);
                        if (SPLIT)
                            P[i] = slice.restored(i, A[i], P[i]);
                    }
                }
            }
        }
    }
    if (SPLIT) {
        put4(seg_at(p.seg_h, p, un, un.seg), kBwdThreads, h);
        put4(seg_at(p.seg_p, p, un, un.seg), kBwdThreads, P);
        put4(seg_at(p.seg_g, p, un, un.seg), kBwdThreads, G);
    }
    ss::pdl_launch_dependents();  // the gradient sweep may take this CTA's place
}

// ------------------------------------------------------------------------- gradient sweep

// The elementwise end of a slice (steps t..t+kT-1, rows r0.. of the stage): a lane has one step of
// its channel pair; and the warp's sums of dB and dC.
template <typename io_t>
__device__ __forceinline__ void finish_slice(const BwdParams& p, const Unit& un, const Cell& x, int t,
                                             int r0, GradSmem<io_t>& sm, const Stage<io_t>& st,
                                             float2& dskip, float2& dbias)
{
    using P2 = Pair<io_t>;
    using raw = typename P2::raw;
#pragma unroll
    for (int step = x.ng; step < kT; step += kG) {
        const int r = r0 + step;
        if (t + step >= un.t1 || !x.valid)
            continue;
        const float2 dl = sm.scal[x.warp][r][0][x.cg], dy = sm.scal[x.warp][r][2][x.cg];
        const float2 u = pair_at(&st.u[r][x.c]);
        auto sum = [&](int q) {
            const float* s = &sm.part[x.warp][q][step][2 * x.cg];
            float2 v[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g)
                v[g] = *reinterpret_cast<const float2*>(s + g * kWC);
#pragma unroll
            for (int m = 1; m < kG; m *= 2)
#pragma unroll
                for (int g = 0; g < kG; g += 2 * m)
                    v[g] = __fadd2_rn(v[g], v[g + m]);
            return v[0];
        };
        const float2 gB = sum(1);
        const float2 gA = __fmul2_rn(sum(2), dup(kLn2));  // A was in base 2
        const float2 skip = again2(&sm.cta.skip[x.c]);
        const float2 du = __ffma2_rn(skip, dy, __fmul2_rn(dl, gB));
        float2 dd = __ffma2_rn(u, gB, gA);
        if (p.softplus)
            dd = __fmul2_rn(dd, sigmoid_2(__fadd2_rn(pair_at(&st.delta[r][x.c]),
                                                  again2(&sm.cta.bias[x.c]))));
        dskip = __ffma2_rn(dy, u, dskip);
        dbias = __fadd2_rn(dbias, dd);
        const uint32_t at = un.row(t + step) + x.c;
        void* out = again(sm.cta.du);
        if (p.du_part)
            *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = du;
        else
            *reinterpret_cast<raw*>(static_cast<io_t*>(out) + at) = P2::r(du);
        *reinterpret_cast<raw*>(static_cast<io_t*>(again(sm.cta.ddelta)) +
                                (static_cast<uint32_t>(t + step) * un.D + x.c)) = P2::r(dd);
        if (p.z) {
            const float2 z = pair_at(&st.z[r][x.c]), sg = sigmoid_2(z);
            const float2 y = __ffma2_rn(skip, u, sum(0));
            // silu'(z) = sg (1 + z (1 - sg))
            const float2 one = dup(1.f), rest = make_float2(1.f - sg.x, 1.f - sg.y);
            const float2 dz = __fmul2_rn(__fmul2_rn(pair_at(&st.dout[r][x.c]), y),
                                         __fmul2_rn(sg, __ffma2_rn(z, rest, one)));
            out = again(sm.cta.dz);
            if (p.dz_part)
                *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = dz;
            else
                *reinterpret_cast<raw*>(static_cast<io_t*>(out) + at) = P2::r(dz);
        }
    }
    // kP lanes add 8 channel pairs each of one (step, tensor, 4 states); lanes of different tensors
    // and parts start at different rows, so that their banks differ
    constexpr int kP = 4 / kG;
    const int n4 = x.lane % kG, q = x.lane / kG & 1, part = x.lane / (2 * kG) % kP, step = x.lane >> 3;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(
            &sm.dbc[x.warp][step][q][8 * part + ((i + 2 * part + q) & 7)][4 * n4]);
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
    }
    if (kP > 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, 4);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, 4);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, 4);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, 4);
    }
    if (part == 0)
        sm.acc[r0 + step][q][x.warp][n4] = v;
}

// dB and dC of a finished tile: the sums of the four warps, to the CTA's partial sums.
template <typename io_t>
__device__ __forceinline__ void store_dbc(const BwdParams& p, const Unit& un, int t, GradSmem<io_t>& sm)
{
    const int rows = min(un.t1 - t, kTL);
    float* out = again(sm.cta.dbc) + static_cast<int64_t>(t) * (2 * kNP);
    constexpr int kVec = 2 * kNP / 4;  // float4 of a step
    for (int j = threadIdx.x; j < rows * kVec; j += kBwdThreads) {
        const int r = j / kVec, q = (j / (kNP / 4)) & 1, n4 = j & (kNP / 4 - 1);
        float4 v = sm.acc[r][q][0][n4];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 a = sm.acc[r][q][w][n4];
            v.x += a.x;
            v.y += a.y;
            v.z += a.z;
            v.w += a.w;
        }
        *reinterpret_cast<float4*>(out + 4 * j) = v;
    }
}

template <typename io_t, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads, 3) grad_kernel(const __grid_constant__ BwdParams p)
{
    constexpr bool PRECISE = std::is_same<io_t, float>::value;
    extern __shared__ __align__(128) unsigned char raw_smem[];
    GradSmem<io_t>& sm = *reinterpret_cast<GradSmem<io_t>*>(raw_smem);
    const Unit un = unit_of(p);
    const Cell x = cell_of(un);
    fill_cta<io_t>(p, un, sm.cta);
    float2 A[4], g[4], dA[4];
    load_A(p, un, x, A);
    float2 dskip = dup(0.f), dbias = dup(0.f);

    const int tiles = (un.t1 - un.t0 + kTL - 1) / kTL;
    io_t bc[kBC][2];
    issue<io_t>(p, un, sm.cta, un.t0 + (tiles - 1) * kTL, sm.st[(tiles - 1) & 1], true, bc);
    ss::pdl_wait();  // from here on the summary sweep's results are read

    // the state that enters the segment and the gradient that enters it from behind
    const bool shift = SPLIT && (un.seg > 0 || p.init != nullptr);
    const int64_t cell = (un.kb * p.D + un.c0 + x.c) * p.N;  // of [K, batch, D, N] arrays
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = 4 * x.ng + i;
        g[i] = dA[i] = dup(0.f);
        if (p.dlast && x.valid && n < p.N)
            g[i] = make_float2(p.dlast[cell + n], p.dlast[cell + p.N + n]);
    }
    if (SPLIT) {
        float2 P[4], v[4], hstart[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * x.ng + i;
            hstart[i] = dup(0.f);
            if (p.init && x.valid && n < p.N)
                hstart[i] = make_float2(p.init[cell + n], p.init[cell + p.N + n]);
        }
#pragma unroll 4
        for (int s = 0; s < un.seg; ++s) {
            get4(seg_at(p.seg_p, p, un, s), kBwdThreads, P);
            get4(seg_at(p.seg_h, p, un, s), kBwdThreads, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                hstart[i] = __ffma2_rn(P[i], hstart[i], v[i]);
        }
        put4(&sm.hstart[0][threadIdx.x], kBwdThreads, hstart);
#pragma unroll 4
        for (int s = p.S - 1; s > un.seg; --s) {
            get4(seg_at(p.seg_p, p, un, s), kBwdThreads, P);
            get4(seg_at(p.seg_g, p, un, s), kBwdThreads, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                g[i] = __ffma2_rn(P[i], g[i], v[i]);
        }
    }

    int slice = (un.t1 - 1) / kT;  // of the sequence; segments start on slice borders
    // the next slice's checkpoint is on its way while this one is worked on
    float2 next[4], next_cum = dup(0.f);
    get4(ckpt_at(un, sm.cta, slice), kBwdThreads, next);
    if (shift && x.valid)
        next_cum = *cum_at(un, sm.cta, x, slice);
    for (int it = tiles - 1; it >= 0; --it) {
        const int t = un.t0 + it * kTL;
        const Stage<io_t>& st = sm.st[it & 1];
        cp_wait_all();
        __syncthreads();
        if (it + 1 < tiles)
            store_dbc(p, un, t + kTL, sm);
        prepass(p, un, x, t, sm, st, true, bc);
        __syncthreads();
        if (it > 0)
            issue<io_t>(p, un, sm.cta, t - kTL, sm.st[(it - 1) & 1], true, bc);

        for (int r0 = kTL - kT; r0 >= 0; r0 -= kT) {
            if (t + r0 >= un.t1)
                continue;
            // the slice's states, from its checkpoint
            float2 h[kT + 1][4], a[kT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[0][i] = next[i];
            if (shift) {
                float2 hstart[4];
                get4(&sm.hstart[0][threadIdx.x], kBwdThreads, hstart);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[0][i] = __ffma2_rn(decay<PRECISE>(next_cum, A[i]), hstart[i], h[0][i]);
            }
            if (t + r0 > un.t0) {
                --slice;
                get4(ckpt_at(un, sm.cta, slice), kBwdThreads, next);
                if (shift && x.valid)
                    next_cum = *cum_at(un, sm.cta, x, slice);
            }
#pragma unroll
            for (int r = 0; r < kT; ++r) {
                float2 B[4];
                load4(sm.B, r0 + r, x.ng, B);
                const float2 dl = sm.scal[x.warp][r0 + r][0][x.cg];
                const float2 w = sm.scal[x.warp][r0 + r][1][x.cg];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[r][i] = decay<PRECISE>(dl, A[i]);
                    h[r + 1][i] = __ffma2_rn(a[r][i], h[r][i], __fmul2_rn(w, B[i]));
                }
            }
            // the reverse recurrence
            Slice slice;
            if (PRECISE)
                slice.start();
#pragma unroll
            for (int r = kT - 1; r >= 0; --r) {
                float2 B[4], C[4], y, gB, gA;
                load4(sm.B, r0 + r, x.ng, B);
                load4(sm.C, r0 + r, x.ng, C);
                const float2 dl = sm.scal[x.warp][r0 + r][0][x.cg];
                const float2 w = sm.scal[x.warp][r0 + r][1][x.cg];
                const float2 dy = sm.scal[x.warp][r0 + r][2][x.cg];
                float dB[4], dC[4];
                if (PRECISE)
                    slice.step(dl);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y = i ? __ffma2_rn(C[i], h[r + 1][i], y) : __fmul2_rn(C[i], h[r + 1][i]);
                    const float2 c2 = __fmul2_rn(dy, h[r + 1][i]);
                    dC[i] = c2.x + c2.y;
                    g[i] = __ffma2_rn(dy, C[i], g[i]);
                    const float2 b2 = __fmul2_rn(w, g[i]);
                    dB[i] = b2.x + b2.y;
                    gB = i ? __ffma2_rn(g[i], B[i], gB) : __fmul2_rn(g[i], B[i]);
                    g[i] = __fmul2_rn(a[r][i], g[i]);
                    if (PRECISE)
                        slice.decayed_by(i, a[r][i]);
                    const float2 q = __fmul2_rn(g[i], h[r][i]);
                    gA = i ? __ffma2_rn(q, A[i], gA) : __fmul2_rn(q, A[i]);
                    dA[i] = __ffma2_rn(q, dl, dA[i]);
                }
                *reinterpret_cast<float2*>(&sm.part[x.warp][0][r][x.ng * kWC + 2 * x.cg]) = y;
                *reinterpret_cast<float2*>(&sm.part[x.warp][1][r][x.ng * kWC + 2 * x.cg]) = gB;
                *reinterpret_cast<float2*>(&sm.part[x.warp][2][r][x.ng * kWC + 2 * x.cg]) = gA;
                *reinterpret_cast<float4*>(&sm.dbc[x.warp][r][0][x.cg][4 * x.ng]) =
                    make_float4(dB[0], dB[1], dB[2], dB[3]);
                *reinterpret_cast<float4*>(&sm.dbc[x.warp][r][1][x.cg][4 * x.ng]) =
                    make_float4(dC[0], dC[1], dC[2], dC[3]);
            }
            if (PRECISE) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    g[i] = slice.restored(i, A[i], g[i]);
            }
            __syncwarp();
            finish_slice(p, un, x, t + r0, r0, sm, st, dskip, dbias);
            __syncwarp();
        }
    }
    __syncthreads();
    store_dbc(p, un, un.t0, sm);

    // what the segment leaves: the initial state's gradient and its parameter gradients
    float* par_out = p.dpar + ((un.kb * p.S + un.seg) * p.D + un.c0 + x.c) * (kNP + 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = 4 * x.ng + i;
        if (x.valid && n < p.N) {
            if (p.g.dinitial_state && un.seg == 0) {
                p.g.dinitial_state[cell + n] = g[i].x;
                p.g.dinitial_state[cell + p.N + n] = g[i].y;
            }
            par_out[n] = dA[i].x;
            par_out[kNP + 2 + n] = dA[i].y;
        }
    }
#pragma unroll
    for (int m = 1; m < kG; m *= 2) {
        dskip.x += __shfl_xor_sync(0xffffffffu, dskip.x, m);
        dskip.y += __shfl_xor_sync(0xffffffffu, dskip.y, m);
        dbias.x += __shfl_xor_sync(0xffffffffu, dbias.x, m);
        dbias.y += __shfl_xor_sync(0xffffffffu, dbias.y, m);
    }
    if (x.ng == 0 && x.valid) {
        par_out[kNP] = dskip.x;
        par_out[kNP + 1] = dbias.x;
        par_out[kNP + 2 + kNP] = dskip.y;
        par_out[kNP + 2 + kNP + 1] = dbias.y;
    }
    ss::pdl_launch_dependents();
}

// ------------------------------------------------------------------------- the last sums

// Blocks [0, bc_blocks): dB, dC = sum over the channel tiles; a thread has one element.
// The next par_blocks x sets: dA, dDskip, ddelta_bias = sum over (direction,) batch rows and
// segments; 32 columns by 8 groups of rows a CTA.
// The rest: du and dz = sum over the directions' parts, four elements a thread.
struct FinishGrid {
    unsigned bc_blocks, par_blocks, sets, dir_blocks;
};

template <typename io_t>
__device__ __forceinline__ void sum_dirs(const float* part, io_t* out, int64_t i, int64_t n, int K)
{
    using P2 = Pair<io_t>;
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

template <typename io_t>
__global__ void __launch_bounds__(256)
    finish_kernel(const __grid_constant__ BwdParams p, const __grid_constant__ FinishGrid grid)
{
    __shared__ float s[8][33];
    ss::pdl_wait();
    unsigned block = blockIdx.x;
    if (block < grid.bc_blocks) {
        const int64_t i = block * int64_t{256} + threadIdx.x;
        const int64_t ctiles = (p.D + kC - 1) / kC;
        if (i >= p.K * p.batch * p.L * 2 * kNP)
            return;
        const int64_t row = i / (2 * kNP);  // kb * L + t
        const int j = static_cast<int>(i % (2 * kNP));
        const int64_t kb = row / p.L, t = row - kb * p.L;
        const float* src = p.dbc + (kb * ctiles * p.L + t) * 2 * kNP + j;
        float v = 0.f;
#pragma unroll 4
        for (int64_t c = 0; c < ctiles; ++c)
            v += src[c * p.L * 2 * kNP];
        const int n = j % kNP;
        if (n < p.N)
            st1(static_cast<io_t*>(j < kNP ? p.g.dB : p.g.dC) + row * p.N + n, v);
        return;
    }
    block -= grid.bc_blocks;
    if (block < grid.par_blocks * grid.sets) {
        const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
        const int64_t cols = p.D * (kNP + 2);
        const int64_t set = block / grid.par_blocks;
        const int64_t col = (block - set * grid.par_blocks) * int64_t{32} + x;
        const int64_t rows = p.K * p.batch * p.S / grid.sets;
        const int64_t d = col / (kNP + 2);
        const int j = static_cast<int>(col - d * (kNP + 2));
        const bool used = col < cols && (j < p.N || j >= kNP);
        float v = 0.f;
        if (used)
#pragma unroll 4
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
        return;
    }
    block -= grid.par_blocks * grid.sets;
    const int64_t n = p.batch * p.L * p.D;  // a multiple of 4
    const int64_t i = 4 * ((block % grid.dir_blocks) * int64_t{256} + threadIdx.x);
    if (i >= n)
        return;
    if (block < grid.dir_blocks && p.du_part)
        sum_dirs(p.du_part, static_cast<io_t*>(p.g.du), i, n, p.K);
    else
        sum_dirs(p.dz_part, static_cast<io_t*>(p.g.dz), i, n, p.K);
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
    e = cudaGetLastError();
    if (e == cudaSuccess)
        e = ss::launch_ex(grad_kernel<io_t, SPLIT>, blocks, kBwdThreads, sizeof(GradSmem<io_t>), st,
                          true, p);
    return e;
}

template <typename io_t> cudaError_t launch_bwd_io(const BwdParams& p, cudaStream_t st)
{
    const cudaError_t e = p.S > 1 || p.init ? launch_sweeps<io_t, true>(p, st)
                                            : launch_sweeps<io_t, false>(p, st);
    if (e != cudaSuccess)
        return e;
    const int64_t nbc = p.K * p.batch * p.L * 2 * kNP, n = p.batch * p.L * p.D;
    FinishGrid g;
    g.bc_blocks = static_cast<unsigned>((nbc + 255) / 256);
    g.par_blocks = static_cast<unsigned>((p.D * (kNP + 2) + 31) / 32);
    g.sets = p.params_per_dir ? p.K : 1;
    g.dir_blocks = static_cast<unsigned>((n / 4 + 255) / 256);
    const unsigned merges = (p.du_part ? 1 : 0) + (p.dz_part ? 1 : 0);
    const unsigned blocks = g.bc_blocks + g.par_blocks * g.sets + g.dir_blocks * merges;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, finish_kernel<io_t>, p, g);
}

}  // namespace

}  // namespace so
