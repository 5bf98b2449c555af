// The selective scan's step for one token per row, on a pool of states that is updated in place.
//
// A step reads and writes 4 N bytes of state per channel and computes 7 operations per state, so
// HBM bounds it for many rows and latency for one.  A warp has 32 channels of a row.  The
// elementwise work (convolution, softplus, gates) runs with one channel a lane.  For the states,
// LPC lanes share a channel with 16-byte accesses (N = 4: 1, N = 8: 2, N = 12 and 16: 4), in LPC
// passes over 32 / LPC channels each, so that every access of a warp is contiguous; Delta and
// Delta u come to the lanes of a channel by shuffle and y goes back the same way.  (With the
// elementwise work done by every lane of a channel the kernel issued 293 instructions for 8 channels
// and was bound by that: 72 us for 256 rows x 5120 channels x 16 states.)  With other N a lane
// has all states of its channel; they, and B and C, pass through shared memory, so that the accesses
// to memory are contiguous there too (directly: N = 15, 111 us for those rows).  A CTA
// keeps its channels' parameters (A alone is as long as a row's state) for up to kRows rows.  Measured
// for those 256 rows, before decays next to one were taken by their distance from it: 42.1 us with 4 rows
// and 24 warps on an SM, 43.3 with 2 rows, 49 with 8; 51 us with 16 warps and the next row's loads ahead
// of the arithmetic.  Now 43.1 us, 68% of the measured HBM rate (N = 15: 59.5).
#include "so_device.cuh"

namespace so {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 4;  // rows of a CTA at most

// Abar h + w of two states, x = Delta A log2(e).  The state is rounded token after token, in place: next
// to one Abar counts by its distance from one, whose relative error is that of the state, where its own
// (2^-22 with the exponential) would be multiplied by the memory.  Series to the fourth power: below
// 1.3e-7 relative at |Delta A| = 1/16, beyond which a memory is 16 tokens at most.  (Not for infinite
// states, which stay.)  Without it, 3000 tokens at memories of 200 to 2000: 4.7e-6 off in the mean, 2.5e-5
// at most; with it 5e-9 and 2.5e-6, at 43.1 us for 41.4 (256 rows x 5120 channels x 16 states).
__device__ __forceinline__ float2 next_state(float2 x, float2 h, float2 w)
{
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    auto two = [](float v) { return make_float2(v, v); };
    float2 c = __ffma2_rn(two(kLn2 * kLn2 * kLn2 * kLn2 / 24.f), x, two(kLn2 * kLn2 * kLn2 / 6.f));
    c = __ffma2_rn(c, x, two(kLn2 * kLn2 / 2.f));
    c = __ffma2_rn(c, x, two(kLn2));
    c = __fmul2_rn(c, x);
    constexpr float kMost = 0.09f;  // 1/16 in base 2
    const bool nx = fabsf(x.x) <= kMost && fabsf(h.x) < __uint_as_float(0x7f800000u);
    const bool ny = fabsf(x.y) <= kMost && fabsf(h.y) < __uint_as_float(0x7f800000u);
    const float2 next = __ffma2_rn(make_float2(nx ? c.x : e.x, ny ? c.y : e.y), h, w);
    return __fadd2_rn(next, make_float2(nx ? h.x : 0.f, ny ? h.y : 0.f));
}

// What a row brings to a lane: the states of its cells, B and C of its state group, and the inputs
// of its channel.
template <typename io_t, int LPC, int NS> struct Row {
    float h[LPC][NS];
    alignas(8) io_t B[4], C[4];  // (N a multiple of 4)
    io_t u, delta, z, seen[SS_MAX_CONV_WIDTH - 1];
};

// UNITS: N / 4, or for an N that is no multiple of 4 the states to make room for, negative.
template <typename io_t, int UNITS>
__global__ void __launch_bounds__(kThreads, UNITS > 0 ? 6 : 3) step_kernel(const StepParams p)
{
    constexpr bool VEC = UNITS > 0;
    constexpr int LPC = UNITS < 2 ? 1 : UNITS == 2 ? 2 : 4;
    constexpr int NS = VEC ? 4 : -UNITS;  // states of a cell
    constexpr int CP = 32 / LPC;                 // channels of a pass
    const int N = VEC ? 4 * UNITS : p.N;
    __shared__ int s_slot[kRows];
    // other N: a warp's states, and B and C of its row
    __shared__ __align__(16) float s_cell[VEC ? 1 : kWarps][VEC ? 4 : 32 * NS];
    __shared__ __align__(16) float s_bc[VEC ? 1 : kWarps][VEC ? 4 : 2 * SS_MAX_DSTATE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = static_cast<int>((p.D + kThreads - 1) / kThreads);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / tiles) * p.rows;
    const int rows = static_cast<int>(p.batch - row0 < p.rows ? p.batch - row0 : p.rows);
    const int64_t d0 = static_cast<int64_t>(blockIdx.x % tiles) * kThreads + warp * 32;
    const int64_t d = d0 + lane;             // the lane's channel in elementwise work
    const int n0 = VEC ? 4 * (lane % LPC) : 0;
    const int nn = VEC ? 4 : N;
    const bool active = d < p.D;
    const int width = p.conv_width;

    // the rows' slots, -1 for padding: a slot outside the pool, or one that an earlier row takes
    for (int r = warp; r < rows; r += kWarps) {
        const int64_t row = row0 + r;
        int slot = static_cast<int>(row);
        if (p.slots) {
            slot = __ldg(p.slots + row);
            int hit = slot < 0 || slot >= p.num_slots;
            for (int64_t i = lane; i < row; i += 32)
                hit |= __ldg(p.slots + i) == slot;
            if (__any_sync(0xffffffffu, hit))
                slot = -1;
        }
        if (lane == 0)
            s_slot[r] = slot;
    }
    // the parameters of the lane's cells and of its channel
    float A[LPC][NS], cw[SS_MAX_CONV_WIDTH], cb = 0.f, skip = 0.f, bias = 0.f;
    bool holds[LPC];
#pragma unroll
    for (int s = 0; s < LPC; ++s) {
        const int64_t c = d0 + s * CP + lane / LPC;
        holds[s] = c < p.D && n0 < N;
#pragma unroll
        for (int n = 0; n < NS; ++n)
            A[s][n] = holds[s] && n < nn ? p.A[c * N + n0 + n] * kLog2e : 0.f;
    }
#pragma unroll
    for (int j = 0; j < SS_MAX_CONV_WIDTH; ++j)
        cw[j] = active && j < width ? p.conv_w[d * width + j] : 0.f;
    if (active) {
        cb = p.conv_b ? p.conv_b[d] : 0.f;
        skip = p.Dskip ? p.Dskip[d] : 0.f;
        bias = p.bias ? p.bias[d] : 0.f;
    }
    __syncthreads();

    // the lane's first cell in slot 0, and the pitches of slots; a pass is CP * N floats further on
    float* const cell0 = p.state + (d0 + lane / LPC) * N + n0;
    const int64_t slot_pitch = p.D * N, window_pitch = p.D * (width - 1);
    io_t* const window0 = static_cast<io_t*>(p.conv_state) + d;
    const int64_t at0 = row0 * p.D + d;  // of [batch, D] tensors
    // other N: the warp's states of a slot as 16-byte pieces (D, and so D * N, is a multiple of 4)
    const int pieces = d0 < p.D ? static_cast<int>(p.D - d0 < 32 ? p.D - d0 : 32) * N / 4 : 0;
    float4* const slot0 = reinterpret_cast<float4*>(p.state + d0 * N);
    float4* const staged = reinterpret_cast<float4*>(s_cell[VEC ? 0 : warp]);
    auto load = [&](int r, Row<io_t, LPC, NS>& x) {
        const int slot = s_slot[r];
        if (slot < 0)
            return;
        const io_t* B = static_cast<const io_t*>(p.B) + (row0 + r) * N + n0;
        const io_t* C = static_cast<const io_t*>(p.C) + (row0 + r) * N + n0;
        if (VEC) {
            const float* cell = cell0 + slot * slot_pitch;
#pragma unroll
            for (int s = 0; s < LPC; ++s)
                if (holds[s]) {
                    const float4 v = *reinterpret_cast<const float4*>(cell + s * CP * N);
                    x.h[s][0] = v.x, x.h[s][1] = v.y, x.h[s][2] = v.z, x.h[s][3] = v.w;
                }
            if (n0 < N) {
                using raw = typename Pair<io_t>::raw;
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    *reinterpret_cast<raw*>(&x.B[n]) = *reinterpret_cast<const raw*>(B + n);
                    *reinterpret_cast<raw*>(&x.C[n]) = *reinterpret_cast<const raw*>(C + n);
                }
            }
        } else {
            const float4* from = slot0 + slot * slot_pitch / 4;
            float4 v[NS / 4];
#pragma unroll
            for (int i = 0; i < NS / 4; ++i)
                if (lane + 32 * i < pieces)
                    v[i] = from[lane + 32 * i];
            const int n = lane % SS_MAX_DSTATE;
            const float bc = n < N ? ld1((lane < SS_MAX_DSTATE ? B : C) + n) : 0.f;
            __syncwarp();  // the row before this one is done with the staged values
#pragma unroll
            for (int i = 0; i < NS / 4; ++i)
                if (lane + 32 * i < pieces)
                    staged[lane + 32 * i] = v[i];
            s_bc[VEC ? 0 : warp][lane] = bc;
        }
        if (active) {
            const int64_t at = at0 + r * p.D;
            x.u = static_cast<const io_t*>(p.u)[at];
            x.delta = static_cast<const io_t*>(p.delta)[at];
            if (p.z)
                x.z = static_cast<const io_t*>(p.z)[at];
            const io_t* win = window0 + slot * window_pitch;
#pragma unroll
            for (int j = 0; j < SS_MAX_CONV_WIDTH - 1; ++j)
                if (j < width - 1)
                    x.seen[j] = win[j * p.D];
        }
    };
    auto step = [&](int r, Row<io_t, LPC, NS>& x) {
        const int slot = s_slot[r];
        if (slot < 0)
            return;  // the same for the whole CTA
        float u = 0.f, delta = 0.f;
        if (active) {
            u = ld1(&x.u);
            if (p.conv_w) {
                float c = cb;
#pragma unroll
                for (int j = 0; j < SS_MAX_CONV_WIDTH - 1; ++j)
                    if (j < width - 1)
                        c = fmaf(cw[j], ld1(&x.seen[j]), c);
                // (constant indices keep the taps in registers)
                c = fmaf(width == 4 ? cw[3] : width == 3 ? cw[2] : width == 2 ? cw[1] : cw[0], u, c);
                if (width > 1) {
                    io_t* win = window0 + slot * window_pitch;
#pragma unroll
                    for (int j = 1; j < SS_MAX_CONV_WIDTH - 1; ++j)
                        if (j < width - 1)
                            win[(j - 1) * p.D] = x.seen[j];
                    win[(width - 2) * p.D] = x.u;
                }
                u = silu_f(c);
            }
            delta = ld1(&x.delta) + bias;
            if (p.softplus)
                delta = softplus_f(delta);
        }
        const float w = delta * u;
        float B[NS], C[NS], y = 0.f;
        if (VEC) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                B[n] = n0 < N ? ld1(&x.B[n % 4]) : 0.f;
                C[n] = n0 < N ? ld1(&x.C[n % 4]) : 0.f;
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                x.h[0][n] = n < nn && active ? s_cell[VEC ? 0 : warp][lane * N + n] : 0.f;
                B[n] = s_bc[VEC ? 0 : warp][n % (2 * SS_MAX_DSTATE)];
                C[n] = s_bc[VEC ? 0 : warp][(SS_MAX_DSTATE + n) % (2 * SS_MAX_DSTATE)];
            }
        }
        float* cell = cell0 + slot * slot_pitch;
#pragma unroll
        for (int s = 0; s < LPC; ++s) {
            // channel s * CP + lane / LPC of the warp, from the lane that has it
            const int from = s * CP + lane / LPC;
            const float dl = LPC > 1 ? __shfl_sync(0xffffffffu, delta, from) : delta;
            const float ws = LPC > 1 ? __shfl_sync(0xffffffffu, w, from) : w;
            float part = 0.f;
            if (holds[s]) {
#pragma unroll
                for (int n = 0; n < NS; n += 2) {
                    float2 v = make_float2(x.h[s][n], x.h[s][n + 1]);
                    const float2 a = make_float2(A[s][n], A[s][n + 1]), d2 = make_float2(dl, dl);
                    v = next_state(__fmul2_rn(a, d2), v, make_float2(ws * B[n], ws * B[n + 1]));
                    x.h[s][n] = v.x, x.h[s][n + 1] = v.y;
                    if (n < nn)
                        part = fmaf(v.x, C[n], part);
                    if (n + 1 < nn)
                        part = fmaf(v.y, C[n + 1], part);
                }
                if (VEC) {
                    *reinterpret_cast<float4*>(cell + s * CP * N) =
                        make_float4(x.h[s][0], x.h[s][1], x.h[s][2], x.h[s][3]);
                } else {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                        if (n < nn)
                            s_cell[VEC ? 0 : warp][lane * N + n] = x.h[s][n];
                }
            }
#pragma unroll
            for (int m = LPC / 2; m > 0; m /= 2)
                part += __shfl_xor_sync(0xffffffffu, part, m);
            // back to the lane of the channel: lane l belongs to pass l / CP
            const float mine = LPC > 1 ? __shfl_sync(0xffffffffu, part, (lane % CP) * LPC) : part;
            y = lane / CP == s ? mine : y;
        }
        if (!VEC) {
            __syncwarp();
            float4* to = slot0 + slot * slot_pitch / 4;
#pragma unroll
            for (int i = 0; i < NS / 4; ++i)
                if (lane + 32 * i < pieces)
                    to[lane + 32 * i] = staged[lane + 32 * i];
        }
        if (active) {
            if (p.Dskip)  // (without, an infinite u would make NaN of y)
                y = fmaf(skip, u, y);
            if (p.z)
                y *= silu_f(ld1(&x.z));
            st1(static_cast<io_t*>(p.out) + at0 + r * p.D, y);
        }
    };
    Row<io_t, LPC, NS> x;
    for (int r = 0; r < rows; ++r) {
        load(r, x);
        step(r, x);
    }
}

template <typename io_t, int UNITS> cudaError_t launch(StepParams p, cudaStream_t st)
{
    const int64_t tiles = (p.D + kThreads - 1) / kThreads;
    // as many rows a CTA as still leave four CTAs for each of 148 SMs
    const int64_t rows = tiles * p.batch / (4 * 148);
    p.rows = static_cast<int>(rows < 1 ? 1 : rows > kRows ? kRows : rows);
    const int64_t blocks = tiles * ((p.batch + p.rows - 1) / p.rows);
    step_kernel<io_t, UNITS><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename io_t> cudaError_t launch_n(const StepParams& p, cudaStream_t st)
{
    if (p.N % 4)
        return p.N < 8 ? launch<io_t, -8>(p, st) : launch<io_t, -SS_MAX_DSTATE>(p, st);
    return p.N == 4    ? launch<io_t, 1>(p, st)
           : p.N == 8  ? launch<io_t, 2>(p, st)
           : p.N == 12 ? launch<io_t, 3>(p, st)
                       : launch<io_t, 4>(p, st);
}

}  // namespace

cudaError_t launch_step(const StepParams& p, int io_dtype, cudaStream_t st)
{
    return io_dtype == SS_BF16 ? launch_n<__nv_bfloat16>(p, st) : launch_n<float>(p, st);
}

}  // namespace so
