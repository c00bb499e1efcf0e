// kvxfer_attn_f16.hip -- attention kernels for half-precision queries, and the choice of type.
#include "kvxfer_attn.h"

namespace kvx {

int launch_attend_bf16(const AttnLaunch &a, int which, bool e4m3, uint32_t grid, hipStream_t stream);
int launch_attend_mx4_f16(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream);
int launch_attend_mx4_bf16(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream);
int launch_join_bf16(const AttnLaunch &a, uint32_t grid, hipStream_t stream);

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

int launch_attend(const AttnLaunch &a, int which, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    const bool half = q_type == KV_TYPE_F16;
    switch (cache_of(kv_type)) {
    case kMx4: return half ? launch_attend_mx4_f16(a, which, grid, stream) : launch_attend_mx4_bf16(a, which, grid, stream);
    case kE4m3:
        return half ? launch_attend_cache<_Float16, kE4m3>(a, which, grid, stream) : launch_attend_bf16(a, which, true, grid, stream);
    default:
        return half ? launch_attend_cache<_Float16, kHalves>(a, which, grid, stream) : launch_attend_bf16(a, which, false, grid, stream);
    }
}

int launch_join(const AttnLaunch &a, int q_type, uint32_t grid, hipStream_t stream)
{
    return q_type == KV_TYPE_F16 ? launch_join_type<_Float16>(a, grid, stream) : launch_join_bf16(a, grid, stream);
}

}  // namespace kvx
