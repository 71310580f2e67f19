// kda_gdn.h -- what the kernels of the gated delta rule with one decay per
// head share.
#pragma once

#include <cudaTypedefs.h>

#include "kda_check.h"
#include "kda_common.cuh"

namespace kda {

struct GdnArgs {
    int Hk, Hv, N, T, num_slots, l2;
    float l2_eps, scale;
    const float* A_log;
    const float* dt_bias;
    const int32_t* cu_seqlens;  // null: sequence s owns row s
    const void* q;
    const void* k;
    const void* v;
    const void* a;
    const void* b;
    long long qs, ks, vs;  // row strides, elements
    const int32_t* slots;
    float* state;
    void* out;
    void* workspace;
    int32_t* dev_status;
};

// The log decay never has to go below this: e^-150 is zero in fp32, 2^-150 too,
// and sums of it over a chunk stay far from the fp32 range (an infinite one
// would make differences of running sums NaN).  NaN passes through.
constexpr float GDN_MIN_LOG = -150.0f;

// ea: e^A_log of the head (times log2 e: the result counts in powers of two).
__device__ __forceinline__ float gdn_log_alpha(float ea, float a, float dt)
{
    const float g = -ea * softplusf_(a + dt);
    return g < GDN_MIN_LOG ? GDN_MIN_LOG : g;
}

// The rows of sequence `seq` and its slot, checked: false (with the fault
// flagged by thread 0 of the CTA) when the unit is skipped.
__device__ __forceinline__ bool gdn_unit(const GdnArgs& a, int seq, int& begin, int& end, int& slot)
{
    begin = seq;
    end = seq + 1;
    if (a.cu_seqlens) {
        begin = a.cu_seqlens[seq];
        end = a.cu_seqlens[seq + 1];
        if (begin < 0 || end < begin || end > a.T) {
            if (threadIdx.x == 0) flag_status(a.dev_status, KDA_DEV_BAD_SEQLENS);
            return false;
        }
    }
    slot = a.slots ? a.slots[seq] : seq;
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) flag_status(a.dev_status, KDA_DEV_BAD_SLOT);
        return false;
    }
    return slot >= 0 && end > begin;
}

// The sequence of rank `rank` by length, longest first (ties: lowest index):
// long chains start first.  More than RANKED sequences balance in any order and keep theirs.
constexpr int RANKED = 128;
__device__ __forceinline__ int ranked_seq(const int32_t* cu, int N, int rank, int* found)
{
    if (N > RANKED || N == 1) return rank;
    const int t = threadIdx.x;
    if (t == 0) *found = rank;
    __syncthreads();
    if (t < N) {
        const int len = cu[t + 1] - cu[t];
        int r = 0;
        for (int i = 0; i < N; ++i) {
            const int l = cu[i + 1] - cu[i];
            r += l > len || (l == len && i < t);
        }
        if (r == rank) *found = t;
    }
    __syncthreads();
    return *found;
}

// The driver's encoder of tensor maps, null where it has none (kda_chunk.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Prefill row by row (fp32 rows), and in chunks on the tensor cores (bf16 rows).
cudaError_t launch_gdn_rows(const GdnArgs& a, int dk, int dv, cudaStream_t st);
cudaError_t launch_gdn_chunk(const GdnArgs& a, int dk, int dv, bool out_bf16, cudaStream_t st);
size_t gdn_chunk_workspace_bytes(int Hk, int Hv, int dk, int N, int T);

}  // namespace kda
