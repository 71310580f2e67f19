// kda_common.cuh -- device helpers shared by the KDA kernels (sm_103a).
//
// Per-row activations of the Kimi Delta Attention layer (ONNX Runtime GenAI
// PR #2843, "Summary of Changes": CausalConvWithState, GatedDeltaNet with
// per-key-dim decay and gate_activation='sigmoid', GatedRMSNorm(activation=
// 'sigmoid'); TensorFold issue #850, Oct 15 comment: conv window, safe or
// softplus gate, beta, q/k L2 norms, delta rule, gated output norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// ------------------------------------------------------------ io types

template <typename T> struct Io;
template <> struct Io<float> {
    static __device__ __forceinline__ float ld(const float* p) { return *p; }
    static __device__ __forceinline__ void st(float* p, float x) { *p = x; }
};
template <> struct Io<__nv_bfloat16> {
    static __device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};

template <typename T> __device__ __forceinline__ float ldv(const T* p) { return Io<T>::ld(p); }
template <typename T> __device__ __forceinline__ void stv(T* p, float x) { Io<T>::st(p, x); }

__device__ __forceinline__ void store_out(void* out, size_t idx, float x, int out_bf16)
{
    if (out_bf16) reinterpret_cast<__nv_bfloat16*>(out)[idx] = __float2bfloat16_rn(x);
    else reinterpret_cast<float*>(out)[idx] = x;
}

// ------------------------------------------------------------ activations
// The same expressions are used by decode, verify and commit so that a
// verified row has the bits of the serially decoded one.

// e^x as 2^(x log2 e) on the special-function unit (PTX ex2.approx.ftz: a
// few ulp; inputs below about -87 give 0, the subnormal results flushed), and
// 1/x by rcp.approx.ftz: one multiply and one SFU instruction each, with no
// range handling around them.
__device__ __forceinline__ float exp_sfu(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__fmul_rn(x, 1.44269504088896341f)));
    return y;
}
__device__ __forceinline__ float exp2_sfu(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_sfu(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoidf_(float x) { return rcp_sfu(__fadd_rn(1.0f, exp_sfu(-x))); }

__device__ __forceinline__ float siluf_(float x) { return __fmul_rn(x, rcp_sfu(__fadd_rn(1.0f, exp_sfu(-x)))); }

// softplus(x) = log(1 + e^x); above 20 the correction e^-x is below fp32
// resolution of x.
__device__ __forceinline__ float softplusf_(float x) { return x > 20.0f ? x : log1pf(exp_sfu(x)); }

// Per-key-dim log decay.  ea = exp(A_log_h).
__device__ __forceinline__ float log_alpha(int gate_mode, float lb, float ea, float f, float dt)
{
    float x = f + dt;
    if (gate_mode == KDA_GATE_SAFE) return lb * sigmoidf_(ea * x);
    return -ea * softplusf_(x);
}

// ------------------------------------------------------------ packed fp32

// two fp32 operations an instruction
__device__ __forceinline__ unsigned long long as_u64(float2 x) { return *reinterpret_cast<unsigned long long*>(&x); }
__device__ __forceinline__ float2 as_f2(unsigned long long x) { return *reinterpret_cast<float2*>(&x); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(r);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ float2 both2(float x) { return make_float2(x, x); }

// ------------------------------------------------------------ tiles of sequences

// Tile c of R rows of a sequence that starts at row `begin` has the number
// begin / R + seq + c: ascending sequences never share one, and there are at
// most T / R + N.  One warp: the sequence of tile x with its rows, or -1 for a
// number without one.  Only sequences within [0, T] are found.  A search of 32
// sequences at a time: 8192 CTAs that each went through 4096 sequences in turn
// would spend longer on that than on their rows.
template <int R>
__device__ __forceinline__ int find_tile(const int32_t* cu, int N, int T, int x, int lane, int& begin, int& end)
{
    int s0 = 0;
    for (int n = (N + 31) / 32; n > 1;) {  // s0 / 32 + 0 .. n - 1: the blocks of 32 sequences left
        const int step = (n + 31) / 32, s = s0 + lane * step * 32;
        const bool below = lane * step < n && min(max(cu[min(s, N)], 0), T) / R + s <= x;
        const int l = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        s0 += l * step * 32;
        n = min(step, n - l * step);
    }
    const int s = s0 + lane;
    begin = s < N ? cu[s] : -1;
    end = s < N ? cu[s + 1] : -1;
    const int c = x - begin / R - s;
    const uint32_t hit = __ballot_sync(0xffffffffu, begin >= 0 && end > begin && end <= T && c >= 0 && c < (end - begin + R - 1) / R);
    if (!hit) return -1;
    const int l = __ffs(hit) - 1;
    begin = __shfl_sync(0xffffffffu, begin, l);
    end = __shfl_sync(0xffffffffu, end, l);
    return s0 + l;
}

// ------------------------------------------------------------ reductions

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void flag_status(int32_t* st, int bit)
{
    if (st) atomicOr(st, bit);
}

// ------------------------------------------------------------ streaming IO

__device__ __forceinline__ float4 ld_stream4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void st_stream4(float* p, float4 v) { __stcs(reinterpret_cast<float4*>(p), v); }

}  // namespace kda
