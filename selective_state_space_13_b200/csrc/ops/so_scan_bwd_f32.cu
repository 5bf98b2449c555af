// Gradient of the selective scan for float io.
#include "so_scan_bwd_kernels.cuh"

namespace so {

cudaError_t launch_scan_bwd_f32(const BwdParams& p, cudaStream_t st)
{
    return launch_bwd_io<float>(p, st);
}

}  // namespace so
