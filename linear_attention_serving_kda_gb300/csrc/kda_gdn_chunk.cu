// kda_gdn_chunk.cu -- the chunked one-decay rule's kernels at dk = 128, the
// workspace's size and the choice by dk (a file for each dk: they compile side
// by side).
#include "kda_gdn_chunk.cuh"

namespace kda {

cudaError_t launch_gdn_chunk_32(const GdnArgs& a, int dv, bool out_bf16, cudaStream_t st);
cudaError_t launch_gdn_chunk_64(const GdnArgs& a, int dv, bool out_bf16, cudaStream_t st);

namespace {

template <int DK> size_t slot_bytes(int Hk, int Hv)
{
    return (size_t)Hk * Slot<DK>::KQ + (size_t)Hv * (Slot<DK>::V + sizeof(int));
}

}  // namespace

size_t gdn_chunk_workspace_bytes(int Hk, int Hv, int dk, int N, int T)
{
    const size_t b = dk == 128 ? slot_bytes<128>(Hk, Hv) : dk == 64 ? slot_bytes<64>(Hk, Hv) : slot_bytes<32>(Hk, Hv);
    return (size_t)slot_count(N, T) * b + sizeof(int);
}

cudaError_t launch_gdn_chunk(const GdnArgs& a, int dk, int dv, bool out_bf16, cudaStream_t st)
{
    if (dk == 128) return out_bf16 ? launch<128, false>(a, dv, st) : launch<128, true>(a, dv, st);
    return dk == 64 ? launch_gdn_chunk_64(a, dv, out_bf16, st) : launch_gdn_chunk_32(a, dv, out_bf16, st);
}

}  // namespace kda
