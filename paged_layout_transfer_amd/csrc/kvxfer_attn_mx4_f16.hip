// kvxfer_attn_mx4_f16.hip -- attention kernels for half-precision queries over 4-bit pools.
#include "kvxfer_attn_mx4.h"

namespace kvx {

int launch_attend_mx4_f16(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream)
{
    return launch_attend_cache<_Float16, kMx4>(a, which, grid, stream);
}

}  // namespace kvx
