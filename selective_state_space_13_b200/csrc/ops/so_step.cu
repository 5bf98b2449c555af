// The selective scan's step for one token per row, on a pool of states that is updated in place.
//
// A step reads and writes 4 N bytes of state per channel and computes 7 operations per state, so
// HBM bounds it for many rows and latency for one.  Four states make one 16-byte access: LPC lanes
// share a channel (N = 4: 1, N = 8: 2, N = 12 and 16: 4), so a warp's state accesses are
// contiguous; other N take one lane per channel and 4-byte accesses, whose lines the next states
// of the same channels find in L1.
#include "so_device.cuh"

namespace so {

namespace {

constexpr int kThreads = 128;

template <typename io_t, int LPC, bool VEC>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepParams p)
{
    constexpr int CH = kThreads / LPC;        // channels of a CTA
    constexpr int NS = VEC ? 4 : SS_MAX_DSTATE;  // states a lane may hold
    const int64_t tiles = (p.D + CH - 1) / CH;
    const int64_t row = blockIdx.x / tiles;
    const int64_t slot = p.slots ? p.slots[row] : row;
    if (slot < 0 || slot >= p.num_slots)
        return;  // the same for the whole CTA
    const int64_t d = (blockIdx.x % tiles) * CH + threadIdx.x / LPC;
    const int n0 = VEC ? 4 * (threadIdx.x % LPC) : 0;
    const int nn = VEC ? 4 : p.N;
    const bool active = d < p.D, holds = active && n0 < p.N;
    float* state = p.state + (slot * p.D + d) * p.N + n0;
    float h[NS], A[NS];
    if (VEC) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), a = v;
        if (holds) {
            v = *reinterpret_cast<const float4*>(state);
            a = make_float4(p.A[d * p.N + n0], p.A[d * p.N + n0 + 1], p.A[d * p.N + n0 + 2],
                            p.A[d * p.N + n0 + 3]);
        }
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        A[0] = a.x, A[1] = a.y, A[2] = a.z, A[3] = a.w;
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            h[n] = holds && n < nn ? state[n] : 0.f;
            A[n] = holds && n < nn ? p.A[d * p.N + n] : 0.f;
        }
    }
    // the inputs before this token; every lane of a channel reads them before one shifts them
    const int width = p.conv_width;
    io_t* win = static_cast<io_t*>(p.conv_state) + slot * (width - 1) * p.D + d;
    io_t seen[SS_MAX_CONV_WIDTH - 1];
#pragma unroll
    for (int j = 0; j < SS_MAX_CONV_WIDTH - 1; ++j)
        if (active && j < width - 1)
            seen[j] = win[j * p.D];
    // the rows before this one decide whether the slot is this row's
    if (p.slots && slot_taken(p.slots, row, static_cast<int32_t>(slot), nullptr, p.batch))
        return;
    __syncwarp();

    float u = 0.f, delta = 0.f, y = 0.f;
    if (active) {
        const io_t* gu = static_cast<const io_t*>(p.u) + row * p.D + d;
        u = ld1(gu);
        if (p.conv_w) {
            const float* cw = p.conv_w + d * width;
            float c = p.conv_b ? p.conv_b[d] : 0.f;
#pragma unroll
            for (int j = 0; j < SS_MAX_CONV_WIDTH - 1; ++j)
                if (j < width - 1)
                    c = fmaf(cw[j], ld1(&seen[j]), c);
            c = fmaf(cw[width - 1], u, c);
            if (threadIdx.x % LPC == 0) {
#pragma unroll
                for (int j = 1; j < SS_MAX_CONV_WIDTH - 1; ++j)
                    if (j < width - 1)
                        win[(j - 1) * p.D] = seen[j];
                if (width > 1)
                    win[(width - 2) * p.D] = *gu;
            }
            u = silu_f(c);
        }
        delta = ld1(static_cast<const io_t*>(p.delta) + row * p.D + d);
        if (p.bias)
            delta += p.bias[d];
        if (p.softplus)
            delta = softplus_f(delta);
    }
    const float w = delta * u, dl = delta * kLog2e;
    const io_t* gB = static_cast<const io_t*>(p.B) + row * p.N + n0;
    const io_t* gC = static_cast<const io_t*>(p.C) + row * p.N + n0;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (holds && n < nn) {
            h[n] = fmaf(ex2(dl * A[n]), h[n], w * ld1(gB + n));
            y = fmaf(h[n], ld1(gC + n), y);
        }
    if (VEC) {
        if (holds)
            *reinterpret_cast<float4*>(state) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (holds && n < nn)
                state[n] = h[n];
    }
#pragma unroll
    for (int m = LPC / 2; m > 0; m /= 2)
        y += __shfl_xor_sync(0xffffffffu, y, m);
    if (active && threadIdx.x % LPC == 0) {
        if (p.Dskip)
            y = fmaf(p.Dskip[d], u, y);
        if (p.z)
            y *= silu_f(ld1(static_cast<const io_t*>(p.z) + row * p.D + d));
        st1(static_cast<io_t*>(p.out) + row * p.D + d, y);
    }
}

template <typename io_t, int LPC, bool VEC> cudaError_t launch(const StepParams& p, cudaStream_t st)
{
    constexpr int CH = kThreads / LPC;
    const int64_t blocks = (p.D + CH - 1) / CH * p.batch;
    step_kernel<io_t, LPC, VEC><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename io_t> cudaError_t launch_n(const StepParams& p, cudaStream_t st)
{
    if (p.N % 4)
        return launch<io_t, 1, false>(p, st);
    return p.N == 4 ? launch<io_t, 1, true>(p, st)
         : p.N == 8 ? launch<io_t, 2, true>(p, st)
                    : launch<io_t, 4, true>(p, st);
}

}  // namespace

cudaError_t launch_step(const StepParams& p, int io_dtype, cudaStream_t st)
{
    return io_dtype == SS_BF16 ? launch_n<__nv_bfloat16>(p, st) : launch_n<float>(p, st);
}

}  // namespace so
