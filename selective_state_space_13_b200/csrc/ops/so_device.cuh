// Device helpers of the operators around the scan: io loads and stores, the elementwise
// functions, and the choice of the row that owns a slot.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "so_internal.h"

namespace so {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ex2.approx errs low: over 2^24 arguments in each decade, the mean of its relative error is
// -0.6e-8 to -2.2e-8 for -0.5 < x < 0 (root mean square 3e-8).  A random error of a decay averages
// out over a state's memory, a mean does not; 2e-8 more in the argument leaves at most 0.8e-8 of it,
// and ex2 of 2e-8 itself is exactly 1, so that a step of zero still keeps the state.  (The scan's
// gradient with bf16 io; the others hold their decays more closely.)
constexpr float kDecayShift = 2e-8f;

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e) for e in [0, 1]: 2 atanh(s), s = e / (2 + e) <= 1/3, as an odd series up to s^15
// (truncation below 2e-9 relative), so that a small e keeps its relative accuracy.
__device__ __forceinline__ float log1p_unit(float e)
{
    const float s = e * rcp(2.f + e);
    const float s2 = s * s;
    float p = fmaf(2.f / 15.f, s2, 2.f / 13.f);
    p = fmaf(p, s2, 2.f / 11.f);
    p = fmaf(p, s2, 2.f / 9.f);
    p = fmaf(p, s2, 2.f / 7.f);
    p = fmaf(p, s2, 2.f / 5.f);
    p = fmaf(p, s2, 2.f / 3.f);
    p = fmaf(p, s2, 2.f);
    return s * p;
}

// softplus(x) = max(x, 0) + log(1 + exp(-|x|)); NaN stays NaN through the exponential.
__device__ __forceinline__ float softplus_f(float x)
{
    return fmaxf(x, 0.f) + log1p_unit(ex2(-fabsf(x) * kLog2e));
}

// 1 / (1 + exp(-x)): both tails keep their relative accuracy (exp overflows to inf, whose
// reciprocal is 0, only where the result is below the normal range).
__device__ __forceinline__ float sigmoid_f(float x) { return rcp(1.f + ex2(-x * kLog2e)); }

__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }

// 1 - exp(x) for x <= 0 (any x): Taylor to x^8 for |x| <= 0.35 (truncation below 8e-10
// relative), so that decays near one keep the relative accuracy of 1 - a.
__device__ __forceinline__ float one_minus_exp(float x, float e)
{
    float p = fmaf(1.f / 40320.f, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p, x, 1.f);
    return fabsf(x) <= 0.35f ? -x * p : 1.f - e;
}

// ---------------------------------------------------------------------------- io types

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two adjacent elements.
template <typename T> struct Pair;
template <> struct Pair<float> {
    using raw = float2;
    static __device__ __forceinline__ float2 f(raw v) { return v; }
    static __device__ __forceinline__ raw r(float2 v) { return v; }
};
template <> struct Pair<__nv_bfloat16> {
    using raw = uint32_t;
    static __device__ __forceinline__ float2 f(raw v)
    {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ raw r(float2 v)
    {
        const __nv_bfloat162 b = __float22bfloat162_rn(v);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
};

// ---------------------------------------------------------------------------- slots

// Whether an earlier row than `row` owns `slot` (all threads of the CTA take part and get the same
// answer): of several rows with one slot only the lowest takes it, so that no two CTAs write the
// same state and the result does not depend on their order.  With `other`, an earlier row counts
// only if its entry there lies in [0, other_slots).
__device__ __forceinline__ bool slot_taken(const int32_t* slots, int64_t row, int32_t slot,
                                           const int32_t* other, int64_t other_slots)
{
    int hit = 0;
    for (int64_t i = threadIdx.x; i < row; i += blockDim.x)
        if (__ldg(slots + i) == slot) {
            const int64_t o = other ? __ldg(other + i) : i;
            hit |= o >= 0 && o < other_slots;
        }
    return __syncthreads_or(hit) != 0;
}

}  // namespace

}  // namespace so
