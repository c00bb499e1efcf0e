// kvxfer_attn_bf16.hip -- attention kernels for bfloat16 queries.
#include "kvxfer_attn.h"

namespace kvx {

int launch_attend_bf16(const AttnLaunch &a, int which, bool e4m3, uint32_t grid, hipStream_t stream)
{
    return launch_attend_type<__bf16>(a, which, e4m3, grid, stream);
}

int launch_join_bf16(const AttnLaunch &a, uint32_t grid, hipStream_t stream)
{
    return launch_join_type<__bf16>(a, grid, stream);
}

}  // namespace kvx
