// kda_gdn_chunk32.cu -- the chunked one-decay rule's kernels at dk = 32.
#include "kda_gdn_chunk.cuh"

namespace kda {

cudaError_t launch_gdn_chunk_32(const GdnArgs& a, int dv, bool out_bf16, cudaStream_t st)
{
    return out_bf16 ? launch<32, false>(a, dv, st) : launch<32, true>(a, dv, st);
}

}  // namespace kda
