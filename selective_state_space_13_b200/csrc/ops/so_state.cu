// Parking of recurrent states in 8 or 4 bits and reading them back: N states of a channel share
// one fp32 scale.  Both directions move bytes and nothing else, so HBM bounds them.  A warp has 32
// channels of a row; where N is a multiple of 4, LPC lanes share a channel with 16-byte state
// accesses in LPC passes (as in the step), and what belongs to a whole channel -- the scale, and in
// the load its codes, 16 bytes for 16 states -- is one lane's; with other N a lane has its channel's
// states and codes from shared memory, through which the warp moves them in contiguous pieces.
//
// round(h q / amax) is what fp32 arithmetic gives wherever its error (below 2^-21 q) cannot move
// the value across the border between two codes; next to a border the quotient is taken again in
// fp64, where h q is exact and the correctly rounded quotient of two fp32 numbers lies on a border
// only if the true one does.  So the codes are those of exact arithmetic.
#include "so_device.cuh"

namespace so {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Pieces of 32 channels that a warp does for one look at the row's slots; their loads are all in
// flight before that look.
constexpr int kChunks = 2;
constexpr int kCtaChannels = kThreads * kChunks;

// The codes of NS states, as bytes; amax is finite and not zero.
template <int NS>
__device__ __forceinline__ void codes_of(const float* h, float amax, int q, uint32_t* code)
{
    // inv is 0 or infinite where q / amax leaves the fp32 range: those go the long way
    const float inv = static_cast<float>(q) * rcp(amax);
    // adding 1.5 * 2^23 leaves the rounded integer in the low bits
    const float2 magic = make_float2(12582912.f, 12582912.f);
    float off = inv > 0.f && inv < 1e30f ? 0.f : 1.f;
#pragma unroll
    for (int n = 0; n < NS; n += 2) {
        const float2 v = __fmul2_rn(make_float2(h[n], h[n + 1]), make_float2(inv, inv));
        const float2 t = __fadd2_rn(v, magic);
        const float2 r = __fadd2_rn(t, make_float2(-magic.x, -magic.y));
        const float2 e = __fadd2_rn(v, make_float2(-r.x, -r.y));  // 1/2 on a border
        off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
        code[n] = __float_as_uint(t.x);
        code[n + 1] = __float_as_uint(t.y);
    }
    if (off > 0.5f - 1e-4f) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            code[n] = static_cast<uint32_t>(
                static_cast<int>(rint(static_cast<double>(h[n]) * q / static_cast<double>(amax))));
    }
}

// Four codes in one unit: 4 bytes, or 4 nibbles with the even states in the low halves.
template <int BITS> struct Unit;
template <> struct Unit<8> {
    using type = uint32_t;
    static __device__ __forceinline__ type pack(const uint32_t* c)
    {
        return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    // the four codes as floats: a byte, its sign bit flipped, in the low bits of 2^23
    static __device__ __forceinline__ float4 get(type v)
    {
        v ^= 0x80808080u;
        auto f = [&](int n) { return __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7540 + n)); };
        const float2 back = make_float2(-8388736.f, -8388736.f);  // -(2^23 + 128)
        const float2 a = __fadd2_rn(make_float2(f(0), f(1)), back);
        const float2 b = __fadd2_rn(make_float2(f(2), f(3)), back);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
template <> struct Unit<4> {
    using type = uint16_t;
    static __device__ __forceinline__ type pack(const uint32_t* c)
    {
        return static_cast<type>((c[0] & 15) | (c[1] & 15) << 4 | (c[2] & 15) << 8 | c[3] << 12);
    }
    static __device__ __forceinline__ float4 get(type v)
    {
        const uint32_t w = v ^ 0x8888u;
        auto f = [&](int n) { return __uint_as_float((w >> (4 * n) & 15u) | 0x4b000000u); };
        const float2 back = make_float2(-8388616.f, -8388616.f);  // -(2^23 + 8)
        const float2 a = __fadd2_rn(make_float2(f(0), f(1)), back);
        const float2 b = __fadd2_rn(make_float2(f(2), f(3)), back);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};

// The row of a CTA: its slots in both pools (false: skipped, the same for the whole CTA), and the
// first channel of the warp.
struct Place {
    int64_t row, src, dst, d0;

    __device__ __forceinline__ bool set(const StateParams& p)
    {
        // (unsigned: a 64-bit division costs as many instructions as the rest of a short kernel)
        const unsigned tiles = (static_cast<unsigned>(p.D) + kCtaChannels - 1) / kCtaChannels;
        const unsigned r = blockIdx.x / tiles;
        row = r;
        d0 = (blockIdx.x - r * tiles) * kCtaChannels + (threadIdx.x >> 5) * 32 * kChunks;
        src = p.src ? p.src[row] : row;
        dst = p.dst ? p.dst[row] : row;
        return src >= 0 && src < p.src_slots && dst >= 0 && dst < p.dst_slots;
    }
};

__device__ __forceinline__ float scale_of(unsigned top, int q)
{
    return top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), static_cast<float>(q))
                             : __uint_as_float(0x7fc00000u);
}

template <int LPC, int BITS>
__global__ void __launch_bounds__(kThreads) store_kernel(const StateParams p)
{
    constexpr int Q = BITS == 8 ? 127 : 7, CP = 32 / LPC;
    using unit_t = typename Unit<BITS>::type;
    Place at;
    if (!at.set(p))
        return;
    const int lane = threadIdx.x & 31, ng = lane % LPC, units = p.N / 4;
    float4 h[kChunks][LPC];
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int s = 0; s < LPC; ++s) {
            const int64_t d = at.d0 + 32 * j + s * CP + lane / LPC;
            h[j][s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (d < p.D && ng < units)
                h[j][s] = reinterpret_cast<const float4*>(p.state_in)[(at.src * p.D + d) * units + ng];
        }
    if (p.dst && slot_taken(p.dst, at.row, static_cast<int32_t>(at.dst), p.src, p.src_slots))
        return;
#pragma unroll
    for (int j = 0; j < kChunks; ++j, at.d0 += 32) {
        unsigned mine = 0;  // the largest magnitude of channel d0 + lane
#pragma unroll
        for (int s = 0; s < LPC; ++s) {
            const float v[4] = {h[j][s].x, h[j][s].y, h[j][s].z, h[j][s].w};
            // by their bits, so that NaN and infinity stand above every number
            unsigned top = 0;
#pragma unroll
            for (int n = 0; n < 4; ++n)
                top = max(top, __float_as_uint(v[n]) & 0x7fffffffu);
#pragma unroll
            for (int m = LPC / 2; m > 0; m /= 2)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
            const unsigned back = LPC > 1 ? __shfl_sync(0xffffffffu, top, (lane % CP) * LPC) : top;
            mine = lane / CP == s ? back : mine;
            uint32_t code[4] = {0, 0, 0, 0};
            if (top - 1 < 0x7f7fffffu)  // neither zero nor infinite nor NaN
                codes_of<4>(v, __uint_as_float(top), Q, code);
            const int64_t d = at.d0 + s * CP + lane / LPC;
            if (d < p.D && ng < units)
                reinterpret_cast<unit_t*>(p.codes)[(at.dst * p.D + d) * units + ng] =
                    Unit<BITS>::pack(code);
        }
        if (at.d0 + lane < p.D)
            p.scales[at.dst * p.D + at.d0 + lane] = scale_of(mine, Q);
    }
}

template <int LPC, int BITS>
__global__ void __launch_bounds__(kThreads) load_kernel(const StateParams p)
{
    constexpr int CP = 32 / LPC;
    using unit_t = typename Unit<BITS>::type;
    struct alignas(sizeof(unit_t) * LPC) Codes {  // of a channel (N = 12: the fourth is unused)
        unit_t v[LPC];
    };
    __shared__ Codes s_codes[kWarps][32];
    Place at;
    if (!at.set(p))
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ng = lane % LPC, units = p.N / 4;
    float scale[kChunks];
    Codes c[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        scale[j] = 0.f;
        c[j] = {};
        if (at.d0 + 32 * j + lane < p.D) {
            const int64_t d = at.src * p.D + at.d0 + 32 * j + lane;
            const unit_t* from = reinterpret_cast<const unit_t*>(p.codes) + d * units;
            scale[j] = p.scales[d];
            if (units == LPC) {
                c[j] = *reinterpret_cast<const Codes*>(from);
            } else {
#pragma unroll
                for (int i = 0; i < LPC; ++i)
                    if (i < units)
                        c[j].v[i] = from[i];
            }
        }
    }
    if (p.dst && slot_taken(p.dst, at.row, static_cast<int32_t>(at.dst), p.src, p.src_slots))
        return;
#pragma unroll
    for (int j = 0; j < kChunks; ++j, at.d0 += 32) {
        __syncwarp();  // the codes before these are read
        s_codes[warp][lane] = c[j];
        __syncwarp();
#pragma unroll
        for (int s = 0; s < LPC; ++s) {
            const int ch = s * CP + lane / LPC;
            const float sc = __shfl_sync(0xffffffffu, scale[j], ch);
            const float4 v = Unit<BITS>::get(s_codes[warp][ch].v[ng]);
            const float2 a = __fmul2_rn(make_float2(v.x, v.y), make_float2(sc, sc));
            const float2 b = __fmul2_rn(make_float2(v.z, v.w), make_float2(sc, sc));
            if (at.d0 + ch < p.D && ng < units)
                reinterpret_cast<float4*>(p.state_out)[(at.dst * p.D + at.d0 + ch) * units + ng] =
                    make_float4(a.x, a.y, b.x, b.y);
        }
    }
}

// n words between memory and shared memory, by a warp, several at a time where both ends allow it.
template <typename word_t, typename wide_t>
__device__ __forceinline__ void move(word_t* dst, const word_t* src, int n, bool wide)
{
    constexpr int W = sizeof(wide_t) / sizeof(word_t);
    const int lane = threadIdx.x & 31;
    if (wide)
        for (int i = lane; i < n / W; i += 32)
            reinterpret_cast<wide_t*>(dst)[i] = reinterpret_cast<const wide_t*>(src)[i];
    else
        for (int i = lane; i < n; i += 32)
            dst[i] = src[i];
}

// Any other N, at most NS: one lane per channel.
template <int BITS, int NS>
__global__ void __launch_bounds__(kThreads) store_any_kernel(const StateParams p)
{
    constexpr int Q = BITS == 8 ? 127 : 7;
    __shared__ __align__(16) float s_state[kWarps][32 * NS];
    __shared__ __align__(16) uint8_t s_codes[kWarps][32 * NS];
    Place at;
    if (!at.set(p))
        return;
    if (p.dst && slot_taken(p.dst, at.row, static_cast<int32_t>(at.dst), p.src, p.src_slots))
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = p.N;
    const int bytes = BITS == 8 ? N : (N + 1) / 2;
    // whole rows start on 16-byte (codes: 4-byte) borders; 32 channels always are a multiple of both
    const bool wide = p.D * N % 4 == 0, wide_codes = p.D * bytes % 4 == 0;
    for (int j = 0; j < kChunks && at.d0 < p.D; ++j, at.d0 += 32) {
        const int count = static_cast<int>(p.D - at.d0 < 32 ? p.D - at.d0 : 32);
        move<float, float4>(s_state[warp], p.state_in + (at.src * p.D + at.d0) * N, count * N, wide);
        __syncwarp();
        float h[NS];
        unsigned top = 0;
        uint32_t code[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            h[n] = n < N && lane < count ? s_state[warp][lane * N + n] : 0.f;
            top = max(top, __float_as_uint(h[n]) & 0x7fffffffu);
            code[n] = 0;
        }
        if (top - 1 < 0x7f7fffffu)
            codes_of<NS>(h, __uint_as_float(top), Q, code);
        if (lane < count) {
            p.scales[at.dst * p.D + at.d0 + lane] = scale_of(top, Q);
#pragma unroll
            for (int i = 0; i < NS * BITS / 8; ++i)
                if (i < bytes)
                    s_codes[warp][lane * bytes + i] = static_cast<uint8_t>(
                        BITS == 8 ? code[i] : (code[2 * i % NS] & 15) | code[(2 * i + 1) % NS] << 4);
        }
        __syncwarp();
        move<uint8_t, uint32_t>(p.codes + (at.dst * p.D + at.d0) * bytes, s_codes[warp], count * bytes,
                                wide_codes);
        __syncwarp();
    }
}

template <int BITS, int NS>
__global__ void __launch_bounds__(kThreads) load_any_kernel(const StateParams p)
{
    __shared__ __align__(16) float s_state[kWarps][32 * NS];
    __shared__ __align__(16) uint8_t s_codes[kWarps][32 * NS];
    Place at;
    if (!at.set(p))
        return;
    if (p.dst && slot_taken(p.dst, at.row, static_cast<int32_t>(at.dst), p.src, p.src_slots))
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = p.N;
    const int bytes = BITS == 8 ? N : (N + 1) / 2;
    const bool wide = p.D * N % 4 == 0, wide_codes = p.D * bytes % 4 == 0;
    for (int j = 0; j < kChunks && at.d0 < p.D; ++j, at.d0 += 32) {
        const int count = static_cast<int>(p.D - at.d0 < 32 ? p.D - at.d0 : 32);
        move<uint8_t, uint32_t>(s_codes[warp], p.codes + (at.src * p.D + at.d0) * bytes, count * bytes,
                                wide_codes);
        const float scale = lane < count ? p.scales[at.src * p.D + at.d0 + lane] : 0.f;
        __syncwarp();
        if (lane < count) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (n < N) {
                    const uint32_t v = s_codes[warp][lane * bytes + n * BITS / 8] >>
                                       (BITS == 4 ? 4 * (n & 1) : 0);
                    s_state[warp][lane * N + n] = (static_cast<int>(v << (32 - BITS)) >> (32 - BITS)) * scale;
                }
        }
        __syncwarp();
        move<float, float4>(p.state_out + (at.dst * p.D + at.d0) * N, s_state[warp], count * N, wide);
        __syncwarp();
    }
}

template <int LPC, int BITS>
cudaError_t launch(const StateParams& p, bool load, cudaStream_t st)
{
    const unsigned blocks = static_cast<unsigned>((p.D + kCtaChannels - 1) / kCtaChannels * p.rows);
    load ? load_kernel<LPC, BITS><<<blocks, kThreads, 0, st>>>(p)
         : store_kernel<LPC, BITS><<<blocks, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int BITS, int NS>
cudaError_t launch_any(const StateParams& p, bool load, cudaStream_t st)
{
    const unsigned blocks = static_cast<unsigned>((p.D + kCtaChannels - 1) / kCtaChannels * p.rows);
    load ? load_any_kernel<BITS, NS><<<blocks, kThreads, 0, st>>>(p)
         : store_any_kernel<BITS, NS><<<blocks, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int BITS> cudaError_t launch_n(const StateParams& p, bool load, cudaStream_t st)
{
    if (p.N % 4)
        return p.N < 8 ? launch_any<BITS, 8>(p, load, st)
                       : launch_any<BITS, SS_MAX_DSTATE>(p, load, st);
    return p.N == 4 ? launch<1, BITS>(p, load, st)
         : p.N == 8 ? launch<2, BITS>(p, load, st)
                    : launch<4, BITS>(p, load, st);
}

}  // namespace

cudaError_t launch_state(const StateParams& p, bool load, cudaStream_t st)
{
    return p.bits == 8 ? launch_n<8>(p, load, st) : launch_n<4>(p, load, st);
}

}  // namespace so
