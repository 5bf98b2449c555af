// Parking of recurrent states in 8 or 4 bits and reading them back: N states of a channel share
// one fp32 scale.  Both directions move bytes and nothing else, so HBM bounds them.  As in the
// step, LPC lanes share a channel with 16-byte state accesses where N is a multiple of 4, and
// other N take one lane per channel.
//
// round(h q / amax) is what fp32 arithmetic gives wherever its error (below 2^-22 q) cannot move
// the value across the border between two codes; next to a border the quotient is taken again in
// fp64, where h q is exact and the correctly rounded quotient of two fp32 numbers lies on a border
// only if the true one does.  So the codes are those of exact arithmetic.
#include "so_device.cuh"

namespace so {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ int code_of(float h, float amax, float inv, int q)
{
    const float v = h * inv;
    const float r = rintf(v);
    // |v - r| is 1/2 on a border; q 2^-22 < 1e-4.  inv is 0 where q / amax leaves the fp32 range.
    if (inv != 0.f && fabsf(fabsf(v - r) - 0.5f) > 1e-4f)
        return static_cast<int>(r);
    return static_cast<int>(rint(static_cast<double>(h) * q / static_cast<double>(amax)));
}

template <int LPC, bool VEC, int BITS>
__global__ void __launch_bounds__(kThreads) store_kernel(const StateParams p)
{
    constexpr int CH = kThreads / LPC, NS = VEC ? 4 : SS_MAX_DSTATE, Q = BITS == 8 ? 127 : 7;
    const int64_t tiles = (p.D + CH - 1) / CH;
    const int64_t row = blockIdx.x / tiles;
    const int64_t src = p.src ? p.src[row] : row, dst = p.dst ? p.dst[row] : row;
    if (src < 0 || src >= p.src_slots || dst < 0 || dst >= p.dst_slots)
        return;  // the same for the whole CTA
    const int64_t d = (blockIdx.x % tiles) * CH + threadIdx.x / LPC;
    const int n0 = VEC ? 4 * (threadIdx.x % LPC) : 0;
    const int nn = VEC ? 4 : p.N;
    const bool active = d < p.D, holds = active && n0 < p.N;
    const float* state = p.state_in + (src * p.D + d) * p.N + n0;
    float h[NS];
    if (VEC) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (holds)
            v = *reinterpret_cast<const float4*>(state);
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            h[n] = holds && n < nn ? state[n] : 0.f;
    }
    if (p.dst && slot_taken(p.dst, row, static_cast<int32_t>(dst), p.src, p.src_slots))
        return;

    // the largest magnitude by its bits, so that NaN and infinity stand above every number
    unsigned top = 0;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        top = max(top, __float_as_uint(h[n]) & 0x7fffffffu);
#pragma unroll
    for (int m = LPC / 2; m > 0; m /= 2)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float amax = __uint_as_float(top);
    const bool fine = top < 0x7f800000u;
    const float scale = fine ? __fdiv_rn(amax, static_cast<float>(Q)) : __uint_as_float(0x7fc00000u);
    const float inv = amax > 1e-30f ? __fdiv_rn(static_cast<float>(Q), amax) : 0.f;
    int code[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n)
        code[n] = fine && top ? code_of(h[n], amax, inv, Q) : 0;
    if (!holds)
        return;
    if (VEC ? threadIdx.x % LPC == 0 : true)
        p.scales[dst * p.D + d] = scale;
    if (BITS == 8) {
        uint8_t* o = p.codes + (dst * p.D + d) * p.N + n0;
        if (VEC) {
            *reinterpret_cast<uchar4*>(o) = make_uchar4(code[0], code[1], code[2], code[3]);
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (n < nn)
                    o[n] = static_cast<uint8_t>(code[n]);
        }
    } else {
        uint8_t* o = p.codes + (dst * p.D + d) * ((p.N + 1) / 2) + n0 / 2;
#pragma unroll
        for (int n = 0; n < NS; n += 2)
            if (n < nn)
                o[n / 2] = static_cast<uint8_t>((code[n] & 15) | (code[n + 1] << 4));
    }
}

template <int LPC, bool VEC, int BITS>
__global__ void __launch_bounds__(kThreads) load_kernel(const StateParams p)
{
    constexpr int CH = kThreads / LPC, NS = VEC ? 4 : SS_MAX_DSTATE;
    const int64_t tiles = (p.D + CH - 1) / CH;
    const int64_t row = blockIdx.x / tiles;
    const int64_t src = p.src ? p.src[row] : row, dst = p.dst ? p.dst[row] : row;
    if (src < 0 || src >= p.src_slots || dst < 0 || dst >= p.dst_slots)
        return;
    const int64_t d = (blockIdx.x % tiles) * CH + threadIdx.x / LPC;
    const int n0 = VEC ? 4 * (threadIdx.x % LPC) : 0;
    const int nn = VEC ? 4 : p.N;
    const bool holds = d < p.D && n0 < p.N;
    int code[NS];
    float scale = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        code[n] = 0;
    if (holds) {
        scale = p.scales[src * p.D + d];
        if (BITS == 8) {
            const int8_t* c = reinterpret_cast<const int8_t*>(p.codes) + (src * p.D + d) * p.N + n0;
            if (VEC) {
                const char4 v = *reinterpret_cast<const char4*>(c);
                code[0] = v.x, code[1] = v.y, code[2] = v.z, code[3] = v.w;
            } else {
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    if (n < nn)
                        code[n] = c[n];
            }
        } else {
            const int8_t* c = reinterpret_cast<const int8_t*>(p.codes) +
                              (src * p.D + d) * ((p.N + 1) / 2) + n0 / 2;
#pragma unroll
            for (int n = 0; n < NS; n += 2)
                if (n < nn) {
                    const int v = c[n / 2];
                    code[n] = static_cast<int8_t>(v << 4) >> 4;
                    code[n + 1] = v >> 4;
                }
        }
    }
    if (p.dst && slot_taken(p.dst, row, static_cast<int32_t>(dst), p.src, p.src_slots))
        return;
    if (!holds)
        return;
    float* state = p.state_out + (dst * p.D + d) * p.N + n0;
    if (VEC) {
        *reinterpret_cast<float4*>(state) =
            make_float4(code[0] * scale, code[1] * scale, code[2] * scale, code[3] * scale);
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (n < nn)
                state[n] = code[n] * scale;
    }
}

template <int LPC, bool VEC, int BITS>
cudaError_t launch(const StateParams& p, bool load, cudaStream_t st)
{
    constexpr int CH = kThreads / LPC;
    const unsigned blocks = static_cast<unsigned>((p.D + CH - 1) / CH * p.rows);
    if (load)
        load_kernel<LPC, VEC, BITS><<<blocks, kThreads, 0, st>>>(p);
    else
        store_kernel<LPC, VEC, BITS><<<blocks, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int BITS> cudaError_t launch_n(const StateParams& p, bool load, cudaStream_t st)
{
    if (p.N % 4)
        return launch<1, false, BITS>(p, load, st);
    return p.N == 4 ? launch<1, true, BITS>(p, load, st)
         : p.N == 8 ? launch<2, true, BITS>(p, load, st)
                    : launch<4, true, BITS>(p, load, st);
}

}  // namespace

cudaError_t launch_state(const StateParams& p, bool load, cudaStream_t st)
{
    return p.bits == 8 ? launch_n<8>(p, load, st) : launch_n<4>(p, load, st);
}

}  // namespace so
