// Gated linear recurrence in one pass over the data.
//
// A column is one batch row and 64 channels; a cluster of CS CTAs walks it together, CS tiles of
// steps at a time.  In a CTA of 4 warps a warp has kSteps consecutive steps of the tile and a lane
// two adjacent channels, so a warp's access is one row of 64 channels.  Every step is the map
// h -> a h + b; a thread composes its steps' maps to a pair (P, H), warp 0 composes the CTA's and,
// through asynchronous stores that count on the receivers' barriers, the cluster's, and then every
// thread runs its steps again from the state they start from, with the decays still in registers.
// So HBM sees every element once; the segments of a split sequence would be read twice.  Each warp
// copies its own rows ahead of their use, which keeps loads in flight while the maps are exchanged.
//
// The gradient is the same recurrence from the last step to the first, q <- a (q + dout).
//
// With so few columns that their clusters leave most of the GPU idle, a long column is cut into
// segments after all: a first launch (`aggregate`) only composes each segment's map, the second
// starts every segment from the maps before it.
//
// A step is a h + w, with a itself: a gate that closes leaves nothing of the old state but a h, and an
// infinite state stays infinite.  Next to a decay of one that would lose 2^-25 of the state (and the
// exponential's error) at every step, which a memory of 1000 steps multiplies.  It does not come to
// that, because states go from one warp's steps to the next through the products P alone, and next to one
// these are taken from U = 1 - P, which is relatively accurate: sigmoid, U' = U + P (1 - a); exp, from the
// sum of the gates.  Where a CTA walks a column alone, as it does in calls of a few steps, the state
// behind its tile is (h - U h) + H, so that token after token loses nothing of a long memory either.
//
// Measured on B200 (8 x 2048 x 1536 bf16): 34.8 us among other passes, 66% of the measured HBM rate.
// With an event around each pass, and a - 1 alone: CTAs of 4 warps, 16 steps a warp, 36.9 us; of 8 warps
// 41 us; of 16 warps with 8 steps 47 us (the barriers cost more than the shorter chains give).  More
// than about three CTAs on an SM run slower, not faster.  TMA boxes for the rows: the same times.
// a - 1 alone, which is wrong where gates close, took 33.0 us among other passes (1 x 131072 x 5120: 731,
// here 756); a = k + m with k = 0 or 1 for every step, as right as this, 39.0 (862); P corrected by what
// every factor had lost, 36.0 (786).
#pragma once

#include <type_traits>

#include "so_device.cuh"
#include "ss_device.cuh"

namespace so {

namespace {

constexpr int kRecWarps = 4;
constexpr int kRecThreads = 32 * kRecWarps;
constexpr int kRecCh = 64;

// Steps of a warp: 16 KB of rows a stage for either type.
template <typename io_t, bool BWD> struct RecTile {
    static constexpr int kTensors = BWD ? 4 : 2;
    static constexpr int kSteps = (BWD ? 16 : 32) / static_cast<int>(sizeof(io_t));
    static constexpr int kRows = kSteps * kRecWarps;
};

template <typename io_t, bool BWD> struct RecSmem {
    using T = RecTile<io_t, BWD>;
    io_t raw[2][T::kTensors][T::kRows][kRecCh];  // [stage][tensor], rows in the order of the steps
    float4 warp_map[kRecWarps][32];  // a warp's steps; then what lies before them in the tile
    float2 start[32];                // the state before the tile
    float2 warp_u[kRecWarps][32];    // U of a warp's steps (a CTA alone)
    float4 cta_map[2][kRecMostCluster][32];  // written by every CTA of the cluster
    uint64_t maps[2];  // the maps of the cluster's CTAs have landed
};

// A decay, and a product of decays, is at least 2^-149 (of a gate of -inf too): that takes a finite
// state below the normal range, and does not make NaN of an infinite one.
constexpr float kLeast = 0x1p-149f;
// The sigmoid's logarithm is at least -125, where 1 + exp(-s) and its reciprocal are normal numbers; what
// is left of the decay there is taken off again (of all: 2^-25 of a decay of 2^-100, less above).
constexpr float kLeastLog2 = -125.f, kLeft = 0x1p-125f - 0x1p-145f;

__device__ __forceinline__ float2 at_least(float2 v, float least)  // (of P: NaN has its say in H)
{
    return make_float2(fmaxf(v.x, least), fmaxf(v.y, least));
}

// The same, and NaN stays.
__device__ __forceinline__ float at_least_nan(float v, float least)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "f"(least));
    return m;
}

// The decays a of two gates and 1 - a, both relatively accurate.  Gate and bias are added before the
// product with log2(e), whose rounding would otherwise be that of the larger one: where 1001 and -1000
// meet, 4e-5 of 1 - a.  The exp form leaves 1 - a out without REST.
template <int FORM, bool REST>
__device__ __forceinline__ void decays_of(float2 gate, float2 bias, float2& a, float2& rest)
{
    const float2 log2e = make_float2(kLog2e, kLog2e), one = make_float2(1.f, 1.f);
    if (FORM == SS_GATE_SIGMOID) {
        const float2 s = __fmul2_rn(__fadd2_rn(gate, bias), log2e);
        const float2 e = make_float2(ex2(-at_least_nan(s.x, kLeastLog2)),
                                     ex2(-at_least_nan(s.y, kLeastLog2)));
        const float2 q = __fadd2_rn(e, one);
        a = make_float2(rcp(q.x), rcp(q.y));
        rest = __fmul2_rn(e, a);
        a = __fadd2_rn(a, make_float2(-kLeft, -kLeft));
    } else {
        const float2 s = __fmul2_rn(gate, log2e);
        a = make_float2(at_least_nan(ex2(s.x), kLeast), at_least_nan(ex2(s.y), kLeast));
        if (REST)
            rest = make_float2(one_minus_exp(gate.x, a.x), one_minus_exp(gate.y, a.y));
    }
}

// U and P of decays whose logarithms add up to `sum`.
__device__ __forceinline__ void product_of_logs(float sum, float& u, float& p)
{
    p = ex2(sum * kLog2e);
    u = one_minus_exp(sum, p);
}

// P from U = 1 - P where that is more accurate.
__device__ __forceinline__ bool near_one(float u) { return fabsf(u) <= 0.5f; }
__device__ __forceinline__ float from_u(float u, float p) { return near_one(u) ? 1.f - u : p; }

// P h + H of one channel, from U where P is near one; an infinite h stays.
__device__ __forceinline__ float through_u(float p, float u, float H, float h)
{
    const bool finite = fabsf(h) < __uint_as_float(0x7f800000u);
    const float next = fmaf(-u, h, H) + h;
    return near_one(u) && finite ? next : fmaf(p, h, H);
}

// 16 bytes global -> shared, zeros where !valid.
__device__ __forceinline__ void cp16(void* dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ss::smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All of this thread's groups of copies but the last have landed.
__device__ __forceinline__ void cp_wait_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_meet()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// Stores v at the place of `p`, an address of this CTA's shared memory, in CTA `rank`'s, and counts
// the 16 bytes on that CTA's barrier `bar`.  No fence is needed on either side: a release at
// cluster scope would wait for the rows that the CTA has stored to HBM.
__device__ __forceinline__ void cluster_store(const float4* p, uint64_t* bar, uint32_t rank, float4 v)
{
    uint32_t at, full;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ss::smem_u32(p)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(full) : "r"(ss::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], "
                 "{%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(full)
                 : "memory");
}

// The map h -> P h + H of two channels, stored as (P.x, P.y, H.x, H.y).
__device__ __forceinline__ float2 through(float4 m, float2 h)
{
    return __ffma2_rn(make_float2(m.x, m.y), h, make_float2(m.z, m.w));
}

// The map f after the map m.
__device__ __forceinline__ float4 compose(float4 f, float4 m)
{
    const float2 P = at_least(__fmul2_rn(make_float2(f.x, f.y), make_float2(m.x, m.y)), kLeast);
    const float2 H = through(f, make_float2(m.z, m.w));
    return make_float4(P.x, P.y, H.x, H.y);
}

// BACK: step s of the recurrence (in the order it runs) lies at position L-1-s.
template <typename io_t, int FORM, bool COMP, bool BWD, bool BACK>
__global__ void __launch_bounds__(kRecThreads, 3)
    recurrence_kernel(const __grid_constant__ RecParams p)
{
    using T = RecTile<io_t, BWD>;
    using P2 = Pair<io_t>;
    using raw = typename P2::raw;
    constexpr int N = T::kSteps;
    extern __shared__ __align__(128) unsigned char raw_smem[];
    RecSmem<io_t, BWD>& sm = *reinterpret_cast<RecSmem<io_t, BWD>*>(raw_smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cs = p.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int ctiles = static_cast<int>((p.D + kRecCh - 1) / kRecCh);
    const int segs = p.aggregate ? p.S - 1 : p.S;  // nobody needs the last one's map
    const int unit = blockIdx.x / cs, column = unit / segs, seg = unit - column * segs;
    const int b = column / ctiles, c0 = (column - b * ctiles) * kRecCh;
    const int d = c0 + 2 * lane;
    const bool active = d < p.D;
    const int L = static_cast<int>(p.L);
    const int t0 = seg * p.seg_len;  // the unit's steps
    const int t1 = L - t0 < p.seg_len ? L : t0 + p.seg_len;
    const int rounds = (t1 - t0 + T::kRows * cs - 1) / (T::kRows * cs);
    const int64_t base = static_cast<int64_t>(b) * p.L * p.D + d;
    float2 bias = make_float2(0.f, 0.f);
    if (p.bias && active)
        bias = make_float2(p.bias[d], p.bias[d + 1]);
    const float* first = BWD ? p.dlast : p.init;
    float2 carry = make_float2(0.f, 0.f);  // the state before this round (kept by warp 0)
    if (first && active)
        carry = make_float2(first[b * p.D + d], first[b * p.D + d + 1]);
    if (cs > 1) {
        if (threadIdx.x == 0) {
            ss::mbar_init(&sm.maps[0], 1);
            ss::mbar_init(&sm.maps[1], 1);
            ss::fence_mbar_init();
        }
        __syncthreads();
        cluster_meet();  // the others' barriers exist
    }
    // A warp copies the rows of its own steps: 16 bytes a lane, whole rows of 64 channels at a time.
    // Channels behind the row and steps behind the end are filled with zeros.
    constexpr int kPiece = 16 / sizeof(io_t), kLanes = kRecCh / kPiece, kAtOnce = 32 / kLanes;
    static_assert(N % kAtOnce == 0, "whole groups of rows");
    const int piece = (lane % kLanes) * kPiece;
    const bool has_piece = c0 + piece < p.D;
    const int64_t from = static_cast<int64_t>(b) * p.L * p.D + c0 + piece;
    auto load = [&](int m) {
        const int first = t0 + (m * cs + rank) * T::kRows + warp * N + lane / kLanes;
        auto rows = [&](int q, const void* tensor, int shift) {
            const io_t* src = static_cast<const io_t*>(tensor) + from;
            io_t* dst = &sm.raw[m & 1][q][warp * N + lane / kLanes][piece];
#pragma unroll
            for (int i = 0; i < N; i += kAtOnce) {
                const int s = first + i + shift;
                const bool ok = has_piece && s < (shift ? L : t1);
                const int64_t at = static_cast<int64_t>(BACK ? L - 1 - s : s) * p.D;
                cp16(dst + i * kRecCh, src + (ok ? at : 0), ok);
            }
        };
        if (m < rounds) {
            rows(0, p.gate, 0);
            if (!BWD) {
                rows(1, p.x, 0);
            } else {
                rows(1, p.dout, 0);
                rows(2, p.out_in, 1);  // the state before a step is the output of the step before it
                if (COMP)
                    rows(T::kTensors - 1, p.x, 0);
            }
        }
        cp_commit();
    };
    load(0);
    if (!BWD)
        load(1);
    // the maps of the segments before this one, which the launch before this one leaves (it may
    // still be running until here); of an aggregate, the product of the decays so far
    float4* const seg_maps = p.seg_maps + static_cast<int64_t>(column) * p.S * 32 + lane;
    float2 product = make_float2(1.f, 1.f);
    if (p.aggregate) {
        carry = make_float2(0.f, 0.f);
    } else if (p.S > 1) {
        ss::pdl_wait();
        if (warp == 0) {
#pragma unroll 4
            for (int s = 0; s < seg; ++s)
                carry = through(seg_maps[s * 32], carry);
        }
    }
    bool waits = true;  // false once a wait has given up: the rest runs without waiting
    const float2 minus = make_float2(-1.f, -1.f), one = make_float2(1.f, 1.f);
    float2 db = make_float2(0.f, 0.f);  // dbias
    for (int m = 0; m < rounds; ++m) {
        const int st = m & 1;
        const int s0 = t0 + (m * cs + rank) * T::kRows + warp * N;  // this warp's first step
        if (BWD) {
            __syncwarp();  // every lane is through with the rows of the round before this one
            load(m + 1);
        }
        cp_wait_one();
        __syncwarp();
        // the thread's two channels of its step i, in tensor q
        const io_t* mine = &sm.raw[st][0][warp * N][2 * lane];
        auto at = [&](int q, int i) {
            return *reinterpret_cast<const raw*>(mine + (q * T::kRows + i) * kRecCh);
        };
        float2 a[N];
        float2 rest[BWD ? N : 1];  // 1 - a
        // what comes in: x, (1 - a) x or dout
        constexpr bool SCALED = COMP && !BWD;
        typename std::conditional<SCALED, float2, raw>::type v[N];
        auto in = [&](int i) {
            if constexpr (SCALED)
                return v[i];
            else
                return P2::f(v[i]);
        };
        float2 P = one, H = make_float2(0.f, 0.f);
        float2 U = make_float2(0.f, 0.f);  // (exp: until the end the sum of the gates)
        // steps behind the end keep the state
        auto compose_steps = [&](bool whole) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 gate = P2::f(at(0, i));
                float2& r = rest[BWD ? i : 0];
                decays_of<FORM, COMP>(gate, bias, a[i], r);
                if constexpr (SCALED)
                    v[i] = __fmul2_rn(r, P2::f(at(1, i)));
                else
                    v[i] = at(1, i);
                const bool inside = whole || s0 + i < t1;
                if (!inside) {
                    a[i] = one;
                    r = make_float2(0.f, 0.f);
                    v[i] = {};
                }
                if (FORM == SS_GATE_SIGMOID)
                    U = __ffma2_rn(r, P, U);
                else if (inside)
                    U = __fadd2_rn(U, gate);
                if (BWD)
                    H = __fmul2_rn(a[i], __fadd2_rn(H, in(i)));
                else
                    H = __ffma2_rn(a[i], H, in(i));
                if (FORM == SS_GATE_SIGMOID)
                    P = __fmul2_rn(a[i], P);
            }
            if (FORM == SS_GATE_EXP) {
                const float2 sum = U;
                product_of_logs(sum.x, U.x, P.x);
                product_of_logs(sum.y, U.y, P.y);
            }
            P = at_least(make_float2(from_u(U.x, P.x), from_u(U.y, P.y)), kLeast);
        };
        const bool whole = s0 + N <= t1;
        if (whole)
            compose_steps(true);
        else
            compose_steps(false);
        sm.warp_map[warp][lane] = make_float4(P.x, P.y, H.x, H.y);
        if (cs == 1)
            sm.warp_u[warp][lane] = U;
        if (!BWD) {
            __syncwarp();  // the rows are in registers: their stage takes those of two rounds on
            load(m + 2);
        }
        __syncthreads();
        if (warp == 0) {
            __syncwarp();
            float4 all = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kRecWarps; ++w) {
                const float4 f = sm.warp_map[w][lane];
                sm.warp_map[w][lane] = all;
                if (cs == 1)
                    U = w ? __ffma2_rn(sm.warp_u[w][lane], make_float2(all.x, all.y), U) : U;
                all = compose(f, all);
            }
            float2 h = carry;
            if (cs > 1) {
                // A CTA sends its map of round m after all its threads are through with the maps of
                // round m - 1, and needs everyone's to go on: the two buffers cannot be overrun.
                if (lane == 0) {
                    ss::mbar_expect_tx(&sm.maps[st], cs * sizeof(sm.cta_map[0][0]));
                    ss::mbar_arrive(&sm.maps[st]);
                }
#pragma unroll
                for (int q = 0; q < kRecMostCluster; ++q)
                    if (q < cs)
                        cluster_store(&sm.cta_map[st][rank][lane], &sm.maps[st], q, all);
                if (waits && !ss::mbar_wait_bounded(&sm.maps[st], (m >> 1) & 1, ss::kWaitLimitNs)) {
                    waits = false;
                    atomicOr(p.status, ss::kStatusTimeout);
                }
#pragma unroll
                for (int q = 0; q < kRecMostCluster; ++q)
                    if (q < cs) {
                        const float4 f = sm.cta_map[st][q][lane];
                        if (q == rank)
                            h = carry;
                        carry = through(f, carry);
                        product = at_least(__fmul2_rn(product, make_float2(f.x, f.y)), kLeast);
                    }
            } else {
                carry = make_float2(through_u(all.x, U.x, all.z, carry.x),
                                    through_u(all.y, U.y, all.w, carry.y));
                product = at_least(__fmul2_rn(product, make_float2(all.x, all.y)), kLeast);
            }
            sm.start[lane] = h;
        }
        __syncthreads();
        if (p.aggregate)
            continue;
        float2 h = through(sm.warp_map[warp][lane], sm.start[lane]);
        // rows of this warp's steps, as byte offsets
        const int64_t stride = (BACK ? -p.D : p.D) * static_cast<int64_t>(sizeof(io_t));
        const int64_t row = (base + static_cast<int64_t>(BACK ? L - 1 - s0 : s0) * p.D) * sizeof(io_t);
        unsigned char* out = static_cast<unsigned char*>(p.out) + row;
        unsigned char* dgate = BWD ? static_cast<unsigned char*>(p.dgate) + row : nullptr;
        auto run_steps = [&](bool whole) {
#pragma unroll
            for (int i = 0; i < N; ++i, out += stride, dgate += BWD ? stride : 0) {
                const bool real = active && (whole || s0 + i < t1);
                if (BWD) {
                    const float2 G = __fadd2_rn(h, in(i));
                    h = __fmul2_rn(a[i], G);
                    float2 before = P2::f(at(2, i));
                    if (s0 + i == L - 1)
                        before = p.init && active
                                     ? make_float2(p.init[b * p.D + d], p.init[b * p.D + d + 1])
                                     : make_float2(0.f, 0.f);
                    if (COMP)
                        before = __ffma2_rn(P2::f(at(T::kTensors - 1, i)), minus, before);
                    float2 ds = __fmul2_rn(h, before);
                    if (FORM == SS_GATE_SIGMOID)
                        ds = __fmul2_rn(ds, rest[i]);
                    if (real) {
                        db = __fadd2_rn(db, ds);
                        *reinterpret_cast<raw*>(out) = P2::r(COMP ? __fmul2_rn(rest[i], G) : G);
                        *reinterpret_cast<raw*>(dgate) = P2::r(ds);
                    }
                } else {
                    h = __ffma2_rn(a[i], h, in(i));
                    if (real)
                        *reinterpret_cast<raw*>(out) = P2::r(h);
                }
            }
        };
        if (whole)
            run_steps(true);
        else if (s0 < t1)
            run_steps(false);
    }
    if (p.aggregate) {
        if (rank == 0 && warp == 0)
            seg_maps[seg * 32] = make_float4(product.x, product.y, carry.x, carry.y);
    } else if (p.last && active && rank == 0 && warp == 0 && seg == p.S - 1) {
        p.last[b * p.D + d] = carry.x;
        p.last[b * p.D + d + 1] = carry.y;
    }
    if (BWD && p.dbias_part && !p.aggregate) {
        __syncthreads();  // the maps are free
        float2* part = reinterpret_cast<float2*>(&sm.warp_map[0][0]);
        part[warp * 32 + lane] = db;
        __syncthreads();
        if (warp == 0 && active) {
#pragma unroll
            for (int w = 1; w < kRecWarps; ++w)
                db = __fadd2_rn(db, part[w * 32 + lane]);
            *reinterpret_cast<float2*>(p.dbias_part + ((static_cast<int64_t>(b) * p.S + seg) * cs + rank) * p.D + d) =
                db;
        }
    }
    ss::pdl_launch_dependents();
    if (cs > 1)
        cluster_meet();  // no CTA leaves while another may store to it
}

template <typename io_t, int FORM, bool COMP, bool BWD, bool BACK>
cudaError_t launch_order(const RecParams& p, cudaStream_t st)
{
    auto kern = recurrence_kernel<io_t, FORM, COMP, BWD, BACK>;
    constexpr int smem = sizeof(RecSmem<io_t, BWD>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t segs = p.aggregate ? p.S - 1 : p.S;
    cfg.gridDim = dim3(static_cast<unsigned>((p.D + kRecCh - 1) / kRecCh * p.batch * segs * p.cluster));
    cfg.blockDim = dim3(kRecThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (p.cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = p.cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (p.S > 1 && !p.aggregate) {  // it may start while the aggregates end
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename io_t, int FORM, bool COMP, bool BWD>
cudaError_t launch_cluster(const RecParams& p, cudaStream_t st)
{
    RecParams q = p;
    for (q.aggregate = p.S > 1 ? 1 : 0; q.aggregate >= 0; --q.aggregate) {
        const cudaError_t e = (p.reverse != 0) != BWD
                                  ? launch_order<io_t, FORM, COMP, BWD, true>(q, st)
                                  : launch_order<io_t, FORM, COMP, BWD, false>(q, st);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace

}  // namespace so
