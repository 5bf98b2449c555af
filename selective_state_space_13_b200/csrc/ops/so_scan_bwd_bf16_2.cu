// Gradient of the selective scan for __nv_bfloat16 io and N up to 8.
#define SO_STATE_GROUPS 2
#include "so_scan_bwd_kernels.cuh"

namespace so {

cudaError_t launch_scan_bwd_bf16_2(const BwdParams& p, cudaStream_t st)
{
    return launch_bwd_io<__nv_bfloat16>(p, st);
}

}  // namespace so
