// kda_paged_f32.cu -- attention of chunks of fp32 rows over a paged cache.
//
// Everything in fp32 on the ordinary pipes (the tensor cores' own fp32 form drops 13 of 24 bits; operands in three bf16 pieces, six products,
// would keep them and were not tried): a CTA holds a tile of R
// rows (all of one key head) and goes through its tokens KEYS at a time: scores S = Q K^T, running maximum and sum of
// each row, O = O 2^(m - m') + W V.  A thread has R / 16 rows x KEYS / 16 scores and the same rows x D / 16 outputs in
// registers, so that a value from shared memory serves four products; two operations an instruction.  The weights take the
// keys' place in shared memory, which leaves room for a second CTA to compute while one loads.
// The multiplications bound it (half of the issue slots, the rest waits for shared memory): 2048 rows of 32 heads of 128 run
// at 39 TFLOP/s, of 256 at 35.
#include "kda_paged_plan.cuh"

namespace kda {
namespace {

using namespace paged;

constexpr int FT = 256;
constexpr int UNIT = 1;
constexpr int ctas_of(int D) { return D == 256 ? 152 : 304; }  // one or two an SM, as shared memory allows

template <int D, int R> struct F32 {
    static constexpr int KEYS = D == 256 ? 32 : 64;
    static constexpr int QS = D + 4, WS = KEYS + 4;  // row strides: 16 rows' same piece in distinct banks
    static constexpr int KW = KEYS * QS > R * WS ? KEYS * QS : R * WS;
    struct Smem {
        float q[R * QS], k[KW], v[KEYS * D];  // k: then the weights
        long long at[KEYS];                   // a token's place in the cache, -1: none, or none that a row sees
    };
};

template <int D, int R> __global__ void __launch_bounds__(FT, D == 256 ? 1 : 2) paged_f32_kernel(const PagedArgs a, const Plan p)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    using L = F32<D, R>;
    constexpr int KEYS = L::KEYS, QS = L::QS, WS = L::WS, RI = R / 16, KI = KEYS / 16, DI = D / 64 > 0 ? D / 64 : 1, DW = D / 16 / DI;
    extern __shared__ __align__(16) unsigned char raw[];
    auto& s = *reinterpret_cast<typename L::Smem*>(raw);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const float c = a.scale * 1.4426950408889634f;
    __shared__ Start start;
    find_start<FT / 32>(a, p, start);
    if (tid == 0) p.cut[blockIdx.x].rows = 0;
    Walk it;
    for (it.start(p, start); it.step(a, p);) {
        if (!it.act) continue;
        const int h = it.head, first = it.lo + it.t0 * KEYS, last = min(it.hi, it.lo + it.t1 * KEYS);
        __syncthreads();
        // A piece without tokens loads no rows: nothing would wait for them before the next piece's rows go to the same place,
        // and of two asynchronous copies to one place either may land last.
        for (int i = tid; first < last && i < R * (D / 4); i += FT) {
            const int r = i / (D / 4), e = i % (D / 4), f = it.row0 + r;
            const bool in = r < it.rows;
            const int tok = group_of(a, f);
            ptx::cp_async16(s.q + r * QS + 4 * e,
                            static_cast<const float*>(a.q) + (in ? (it.begin + tok) * a.q_stride + (long long)(h * a.G + f - tok * a.G) * D + 4 * e : 0), in ? 16 : 0);
        }
        float m[RI], l[RI];
        float2 o[RI][DI][DW / 2];
        int pos[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            pos[i] = it.pos0() + group_of(a, it.row0 + ty + 16 * i);
#pragma unroll
            for (int d = 0; d < DI; ++d)
#pragma unroll
                for (int e = 0; e < DW / 2; ++e) o[i][d][e] = make_float2(0.f, 0.f);
        }
        for (int k0 = first; k0 < last; k0 += KEYS) {
            __syncthreads();  // the tile before is done with
            if (tid < KEYS) {
                const int t = k0 + tid;
                long long at = -1;
                // (the first token that a row sees, from the rows: it.seen kept over the loop costs registers, 885 us for 874)
                if (t < last && !(a.window && t <= it.pos0() + group_of(a, it.row0) - (long long)a.window)) {
                    const int page = a.pages[(long long)it.seq * a.width + (t >> a.page_shift)];
                    if (page < 0 || page >= a.num_pages) flag_status(a.dev_status, KDA_DEV_BAD_PAGE);
                    else at = page * a.page_stride + (t & ((1 << a.page_shift) - 1)) * a.token_stride + h * a.head_stride;
                }
                s.at[tid] = at;
            }
            __syncthreads();
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // keys first: they are needed first
                const float* src = static_cast<const float*>(half ? a.v : a.k);
                float* dst = half ? s.v : s.k;
                const int stride = half ? D : QS;
                for (int i = tid; i < KEYS * (D / 4); i += FT) {
                    const int t = i / (D / 4), e = i % (D / 4);
                    const long long at = s.at[t];
                    ptx::cp_async16(dst + t * stride + 4 * e, src + (at >= 0 ? at + 4 * e : 0), at >= 0 ? 16 : 0);
                }
                ptx::cp_async_commit();
            }
            ptx::cp_async_wait_prev();
            __syncthreads();
            float2 w[RI][KI];
#pragma unroll
            for (int i = 0; i < RI; ++i)
#pragma unroll
                for (int j = 0; j < KI; ++j) w[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int e = 0; e < D; e += 4) {
                float4 q[RI], k[KI];
#pragma unroll
                for (int i = 0; i < RI; ++i) q[i] = *reinterpret_cast<const float4*>(s.q + (ty + 16 * i) * QS + e);
#pragma unroll
                for (int j = 0; j < KI; ++j) k[j] = *reinterpret_cast<const float4*>(s.k + (tx + 16 * j) * QS + e);
#pragma unroll
                for (int i = 0; i < RI; ++i)
#pragma unroll
                    for (int j = 0; j < KI; ++j)
                        w[i][j] = fma2(make_float2(q[i].z, q[i].w), make_float2(k[j].z, k[j].w), fma2(make_float2(q[i].x, q[i].y), make_float2(k[j].x, k[j].y), w[i][j]));
            }
            __syncthreads();  // the keys are read: their place takes the weights
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                float x[KI], most = -INFINITY;
#pragma unroll
                for (int j = 0; j < KI; ++j) {
                    const int t = k0 + tx + 16 * j;
                    const bool seen = s.at[tx + 16 * j] >= 0 && (!a.causal || (t <= pos[i] && (!a.window || t > pos[i] - (long long)a.window)));
                    x[j] = seen ? (w[i][j].x + w[i][j].y) * c : -INFINITY;
                    most = fmaxf(most, x[j]);
                }
#pragma unroll
                for (int x2 = 8; x2 > 0; x2 >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x2));
                const float next = fmaxf(m[i], most), base = next == -INFINITY ? 0.f : next;
                const float f = exp2f(m[i] - base);
                m[i] = next;
                l[i] *= f;
#pragma unroll
                for (int j = 0; j < KI; ++j) {
                    const float y = exp2f(x[j] - base);
                    l[i] += y;
                    s.k[(ty + 16 * i) * WS + tx + 16 * j] = y;
                }
#pragma unroll
                for (int d = 0; d < DI; ++d)
#pragma unroll
                    for (int e = 0; e < DW / 2; ++e) o[i][d][e] = mul2(o[i][d][e], both2(f));
            }
            ptx::cp_async_wait_all();
            __syncthreads();
#pragma unroll 2
            for (int t = 0; t < KEYS; t += 4) {
                float4 y[RI];
#pragma unroll
                for (int i = 0; i < RI; ++i) y[i] = *reinterpret_cast<const float4*>(s.k + (ty + 16 * i) * WS + t);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float2 v[DI][DW / 2];
#pragma unroll
                    for (int d = 0; d < DI; ++d) {
                        const float* x = s.v + (t + u) * D + d * 64 + tx * DW;
                        if constexpr (DW == 4) {
                            const float4 z = *reinterpret_cast<const float4*>(x);
                            v[d][0] = make_float2(z.x, z.y);
                            v[d][DW / 2 - 1] = make_float2(z.z, z.w);
                        } else {
                            v[d][0] = *reinterpret_cast<const float2*>(x);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < RI; ++i) {
                        const float2 yy = both2(u == 0 ? y[i].x : u == 1 ? y[i].y : u == 2 ? y[i].z : y[i].w);
#pragma unroll
                        for (int d = 0; d < DI; ++d)
#pragma unroll
                            for (int e = 0; e < DW / 2; ++e) o[i][d][e] = fma2(yy, v[d][e], o[i][d][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
#pragma unroll
            for (int x2 = 8; x2 > 0; x2 >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x2);
            const int r = ty + 16 * i, f = it.row0 + r, tok = group_of(a, f);
            if (r >= it.rows) continue;
            const size_t row = (size_t)(it.begin + tok) * a.Hq + h * a.G + f - tok * a.G;
            const size_t cell = (size_t)blockIdx.x * 2 + (it.t0 == 0);
            const bool whole = it.whole(), none = l[i] == 0.f;
            const float2 inv = both2(!whole ? 1.f : none ? 0.f : 1.f / l[i]);
#pragma unroll
            for (int d = 0; d < DI; ++d)
#pragma unroll
                for (int e = 0; e < DW / 2; ++e) {
                    const float2 y = none ? make_float2(0.f, 0.f) : mul2(o[i][d][e], inv);
                    const int ch = d * 64 + tx * DW + 2 * e;
                    if (whole) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + ch) = y;
                    else reinterpret_cast<float2*>(p.o + (cell * (D / 4) + ch / 4) * p.part_rows + r)[ch % 4 / 2] = y;
                }
            if (tx == 0) {
                if (!whole) p.ml[cell * p.part_rows + r] = make_float2(m[i], l[i]);
                else if (a.lse) a.lse[row] = none ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
            }
        }
        if (tid == 0 && it.t0 == 0 && !it.whole()) p.cut[blockIdx.x] = {start.line, it.begin, it.row0, it.rows, h, owner(start.line, it.end(p) - 1, p.ctas)};
    }
    ptx::cp_async_wait_all();
}

// Rows of a tile: 16 where sequences have that few (a token or two of the group's heads), else 64.
int tile_rows(const PagedArgs& a) { return (int64_t)a.T * a.G <= 16 * (int64_t)a.N ? 16 : 64; }

template <int D, int R> cudaError_t launch(const PagedArgs& a, cudaStream_t st)
{
    using L = F32<D, R>;
    constexpr int smem = sizeof(typename L::Smem);
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(paged_f32_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    Plan p;
    lay_out(p, a, R, L::KEYS, ctas_of(D), UNIT);
    e = launch_dependent(paged_f32_kernel<D, R>, ctas_of(D), FT, smem, st, a, p);
    if (e == cudaSuccess) e = launch_join<float, D>(a, p, st);
    return e;
}

template <int D> cudaError_t launch_rows(const PagedArgs& a, cudaStream_t st)
{
    return tile_rows(a) == 16 ? launch<D, 16>(a, st) : launch<D, 64>(a, st);
}

}  // namespace

size_t paged_f32_workspace_bytes(const PagedArgs& a)
{
    Plan p;
    return lay_out(p, a, tile_rows(a), a.D == 256 ? 32 : 64, ctas_of(a.D), 0);
}

cudaError_t launch_paged_f32(const PagedArgs& a, cudaStream_t st)
{
    switch (a.D) {
    case 32: return launch_rows<32>(a, st);
    case 64: return launch_rows<64>(a, st);
    case 128: return launch_rows<128>(a, st);
    default: return launch_rows<256>(a, st);
    }
}

}  // namespace kda
