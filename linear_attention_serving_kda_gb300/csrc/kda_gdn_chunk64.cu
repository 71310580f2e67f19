// kda_gdn_chunk64.cu -- the chunked one-decay rule's kernels at dk = 64.
#include "kda_gdn_chunk.cuh"

namespace kda {

cudaError_t launch_gdn_chunk_64(const GdnArgs& a, int dv, bool out_bf16, cudaStream_t st)
{
    return out_bf16 ? launch<64, false>(a, dv, st) : launch<64, true>(a, dv, st);
}

}  // namespace kda
