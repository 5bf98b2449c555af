// Gated linear recurrence and its gradient: the launches.
#include "so_recurrence_cluster.cuh"

namespace so {

namespace {

// out[d] = sum over rows of part[row, d], in a fixed order: 32 channels by 8 row groups a CTA.
struct SumRows {
    const float* part;
    float* out;
    int64_t rows, D;
};

__global__ void __launch_bounds__(256) sum_rows_kernel(const SumRows p)
{
    __shared__ float s[8][33];
    ss::pdl_wait();  // the launch before this one writes the rows
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t d = blockIdx.x * int64_t{32} + x;
    float v = 0.f;
    if (d < p.D)
        for (int64_t r = y; r < p.rows; r += 8)
            v += p.part[r * p.D + d];
    s[y][x] = v;
    __syncthreads();
    if (y == 0 && d < p.D) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v += s[i][x];
        p.out[d] = v;
    }
}

template <typename io_t, int FORM, bool COMP>
cudaError_t launch(const RecParams& p, bool backward, cudaStream_t st)
{
    if (!backward)
        return launch_cluster<io_t, FORM, COMP, false>(p, st);
    cudaError_t e = launch_cluster<io_t, FORM, COMP, true>(p, st);
    if (e == cudaSuccess && p.dbias) {
        const SumRows s = {p.dbias_part, p.dbias, p.batch * p.S * p.cluster, p.D};
        e = ss::launch_ex(sum_rows_kernel, static_cast<unsigned>((p.D + 31) / 32), 256, 0, st, true, s);
    }
    return e;
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

int recurrence_tile(int io_dtype, bool backward)
{
    if (io_dtype == SS_BF16)
        return backward ? RecTile<__nv_bfloat16, true>::kRows : RecTile<__nv_bfloat16, false>::kRows;
    return backward ? RecTile<float, true>::kRows : RecTile<float, false>::kRows;
}

}  // namespace so
