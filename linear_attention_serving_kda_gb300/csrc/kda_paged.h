// kda_paged.h -- what the kernels of softmax attention over a paged cache share.
#pragma once

#include <cudaTypedefs.h>

#include "kda_check.h"
#include "kda_common.cuh"

namespace kda {

struct PagedArgs {
    int Hq, Hkv, G, D, N, T;
    uint32_t g_mul;  // with g_shift: division by G (group_of)
    int g_shift;
    int page_shift, num_pages, width;  // width: entries of a sequence's row of `pages`
    int causal, window;
    float scale;
    long long page_stride, token_stride, head_stride, q_stride;  // elements
    const int32_t* cu_seqlens;  // null: sequence s owns row s
    const int32_t* kv_lens;
    const int32_t* pages;
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;
    void* workspace;
    int32_t* dev_status;
    uint32_t polls, unit_polls;  // after which a wait gives up: for a tile, for 2^16 tiles of a unit
    int stalled;                 // the CTA that loads nothing, -1: none (kda_debug_paged_attn_stalled)
};

constexpr uint32_t PAGED_POLLS = 1u << 22;
// Sum of the weights of a part, or of a warp's share of one, whose waits gave up: there is no other value below zero.  The joins leave its rows out.
constexpr float PART_LOST = -1.f;

// n / G for 0 <= n < 2^31, as n M / 2^(31 + s) with 2^(s - 1) < G <= 2^s and M = floor(2^(31 + s) / G) + 1: M G is above
// 2^(31 + s) by at most G <= 2^s, which makes less than n 2^s / (G 2^(31 + s)) < 1 / G of difference, too little to reach the next quotient.
__device__ __forceinline__ int group_of(const PagedArgs& a, int n) { return (int)(((uint64_t)(uint32_t)n * a.g_mul) >> a.g_shift); }

// Tokens that a row of the table can name.
__device__ __forceinline__ long long paged_capacity(const PagedArgs& a) { return (long long)a.width << a.page_shift; }

// The rows begin .. end - 1 of sequence s and its tokens, checked; false when it is skipped (with
// the fault in *fault).
__device__ __forceinline__ bool paged_seq(const PagedArgs& a, int s, int& begin, int& end, int& kv, int* fault)
{
    begin = s;
    end = s + 1;
    kv = a.kv_lens[s];
    if (a.cu_seqlens) {
        begin = a.cu_seqlens[s];
        end = a.cu_seqlens[s + 1];
        if (begin < 0 || end < begin || end > a.T) {
            *fault |= KDA_DEV_BAD_SEQLENS;
            return false;
        }
    }
    if (kv > paged_capacity(a)) {
        *fault |= KDA_DEV_BAD_SEQLENS;
        return false;
    }
    return kv >= 0 && end > begin;
}

// Attention of chunks: fp32 rows, bf16 rows; of single tokens, where `wanted`.
cudaError_t launch_paged_f32(const PagedArgs& a, cudaStream_t st);
size_t paged_f32_workspace_bytes(const PagedArgs& a);
cudaError_t launch_paged_bf16(const PagedArgs& a, cudaStream_t st);
size_t paged_bf16_workspace_bytes(const PagedArgs& a);
cudaError_t launch_paged_token(const PagedArgs& a, bool f32, cudaStream_t st);
size_t paged_token_workspace_bytes(const PagedArgs& a);
bool paged_token_wanted(const PagedArgs& a, bool f32);

// The driver's encoder of tensor maps, null where it has none (kda_chunk.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace kda
