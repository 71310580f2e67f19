// kda_check.h -- host-side argument checks shared by the C entry points.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "kda_internal.h"

namespace kda {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int io_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }
inline bool known_dtype(int dtype) { return dtype == KDA_DTYPE_F32 || dtype == KDA_DTYPE_BF16; }

// Every pointer in the list must be non-null and 16-byte aligned.
inline int check_ptrs(std::initializer_list<const void*> ps)
{
    for (const void* x : ps)
        if (!x || !aligned16(x)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

inline int check_opt(const void* x) { return (x && !aligned16(x)) ? KDA_ERR_INVALID_ARGUMENT : KDA_OK; }

// Whether [a, a + na) and [b, b + nb) share a byte (null: no).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Launches a kernel that may begin before the one ahead of it on the stream has
// ended (programmatic dependent launch): every thread of it waits for that end
// (ptx::grid_dependency_wait) before its first access to memory.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// KDA_OK on an sm_103 device (the answer is remembered per device).
int check_device();
// SMs of the current device, 0 when it cannot be asked.
int sm_count();
// SMs that kernels on the stream may use: fewer than the device's where the stream belongs to a partition of it
// (a green context), 0 where the driver does not say.
int stream_sm_count(cudaStream_t stream);

}  // namespace kda
