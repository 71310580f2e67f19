// kda_paged_f32.cu -- attention over a paged cache for fp32 rows, chunks and single tokens.
//
// Everything in fp32 on the ordinary pipes: a CTA holds a tile of R rows (all of one key head) and goes
// through its tokens KEYS at a time: scores S = Q K^T, running maximum and sum of each row, O = O 2^(m - m') + W V.
// A thread has R / 16 rows x KEYS / 16 scores and the same rows x D / 16 outputs in registers, so that a value from
// shared memory serves 4 products.
#include "kda_paged_plan.cuh"

namespace kda {
namespace {

using namespace paged;

constexpr int FT = 256;
constexpr int CTAS = 304;  // two an SM

template <int D, int R> struct F32 {
    static constexpr int KEYS = D == 256 ? 32 : 64;
    static constexpr int QS = D + 4, WS = KEYS + 4;  // row strides: 16 rows' same piece in distinct banks
    struct Smem {
        float q[R * QS], k[KEYS * QS], v[KEYS * D], w[R * WS];
        long long at[KEYS];  // a token's place in the cache, -1: none
    };
};

template <typename IO> __device__ __forceinline__ float4 load4(const void* base, long long at)
{
    const IO* x = static_cast<const IO*>(base) + at;
    if constexpr (sizeof(IO) == 4) return *reinterpret_cast<const float4*>(x);
    else return make_float4(ldv(x), ldv(x + 1), ldv(x + 2), ldv(x + 3));
}

template <typename IO, int D, int R> __global__ void __launch_bounds__(FT) paged_f32_kernel(const PagedArgs a, const Plan p)
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
    for (it.begin_at(a, p, start); it.left > 0; it.next(a, p)) {
        if (!it.act) continue;
        const int h = it.head, first = it.lo + it.t0 * KEYS, last = min(it.hi, it.lo + it.t1 * KEYS);
        __syncthreads();
        for (int i = tid; i < R * (D / 4); i += FT) {
            const int r = i / (D / 4), e = i % (D / 4), f = it.row0 + r;
            float4 q = make_float4(0, 0, 0, 0);
            if (r < it.rows)
                q = load4<IO>(a.q, (it.begin + f / a.G) * a.q_stride + (long long)(h * a.G + f % a.G) * D + 4 * e);
            *reinterpret_cast<float4*>(s.q + r * QS + 4 * e) = q;
        }
        float m[RI], l[RI], o[RI][DI][DW];
        int pos[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            pos[i] = it.pos0() + (it.row0 + ty + 16 * i) / a.G;
#pragma unroll
            for (int d = 0; d < DI; ++d)
#pragma unroll
                for (int e = 0; e < DW; ++e) o[i][d][e] = 0.f;
        }
        for (int k0 = first; k0 < last; k0 += KEYS) {
            __syncthreads();  // the tile before is done with
            if (tid < KEYS) {
                const int t = k0 + tid;
                long long at = -1;
                if (t < last) {
                    const int page = a.pages[(long long)it.seq * a.width + (t >> a.page_shift)];
                    if (page < 0 || page >= a.num_pages) flag_status(a.dev_status, KDA_DEV_BAD_PAGE);
                    else at = page * a.page_stride + (t & ((1 << a.page_shift) - 1)) * a.token_stride + h * a.head_stride;
                }
                s.at[tid] = at;
            }
            __syncthreads();
            for (int i = tid; i < KEYS * (D / 4); i += FT) {
                const int t = i / (D / 4), e = i % (D / 4);
                const long long at = s.at[t];
                float4 k = make_float4(0, 0, 0, 0), v = k;
                if (at >= 0) {
                    k = load4<IO>(a.k, at + 4 * e);
                    v = load4<IO>(a.v, at + 4 * e);
                }
                *reinterpret_cast<float4*>(s.k + t * QS + 4 * e) = k;
                *reinterpret_cast<float4*>(s.v + t * D + 4 * e) = v;
            }
            __syncthreads();
            float w[RI][KI];
#pragma unroll
            for (int i = 0; i < RI; ++i)
#pragma unroll
                for (int j = 0; j < KI; ++j) w[i][j] = 0.f;
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
                        w[i][j] = fmaf(q[i].w, k[j].w, fmaf(q[i].z, k[j].z, fmaf(q[i].y, k[j].y, fmaf(q[i].x, k[j].x, w[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                float most = -INFINITY;
#pragma unroll
                for (int j = 0; j < KI; ++j) {
                    const int t = k0 + tx + 16 * j;
                    const bool seen = s.at[tx + 16 * j] >= 0 && (!a.causal || (t <= pos[i] && (!a.window || t > pos[i] - (long long)a.window)));
                    w[i][j] = seen ? w[i][j] * c : -INFINITY;
                    most = fmaxf(most, w[i][j]);
                }
#pragma unroll
                for (int x2 = 8; x2 > 0; x2 >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x2));
                const float next = fmaxf(m[i], most), base = next == -INFINITY ? 0.f : next;
                const float f = exp2f(m[i] - base);
                m[i] = next;
                l[i] *= f;
#pragma unroll
                for (int j = 0; j < KI; ++j) {
                    const float y = exp2f(w[i][j] - base);
                    l[i] += y;
                    s.w[(ty + 16 * i) * WS + tx + 16 * j] = y;
                }
#pragma unroll
                for (int d = 0; d < DI; ++d)
#pragma unroll
                    for (int e = 0; e < DW; ++e) o[i][d][e] *= f;
            }
            __syncwarp();  // a row's weights come from and go to its half of the warp
#pragma unroll 2
            for (int t = 0; t < KEYS; t += 4) {
                float4 y[RI];
#pragma unroll
                for (int i = 0; i < RI; ++i) y[i] = *reinterpret_cast<const float4*>(s.w + (ty + 16 * i) * WS + t);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float v[DI][DW];
#pragma unroll
                    for (int d = 0; d < DI; ++d)
#pragma unroll
                        for (int e = 0; e < DW; ++e) v[d][e] = s.v[(t + u) * D + d * 64 + tx * DW + e];
#pragma unroll
                    for (int i = 0; i < RI; ++i) {
                        const float yy = u == 0 ? y[i].x : u == 1 ? y[i].y : u == 2 ? y[i].z : y[i].w;
#pragma unroll
                        for (int d = 0; d < DI; ++d)
#pragma unroll
                            for (int e = 0; e < DW; ++e) o[i][d][e] = fmaf(yy, v[d][e], o[i][d][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
#pragma unroll
            for (int x2 = 8; x2 > 0; x2 >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x2);
            const int r = ty + 16 * i, f = it.row0 + r;
            if (r >= it.rows) continue;
            const size_t row = (size_t)(it.begin + f / a.G) * a.Hq + h * a.G + f % a.G;
            const size_t cell = (size_t)blockIdx.x * 2 + (it.t0 == 0);
            const bool whole = it.whole();
            const float inv = !whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
            for (int d = 0; d < DI; ++d)
#pragma unroll
                for (int e = 0; e < DW; ++e) {
                    const float y = l[i] == 0.f ? 0.f : o[i][d][e] * inv;
                    if (whole) stv(static_cast<IO*>(a.out) + row * D + d * 64 + tx * DW + e, y);
                    else reinterpret_cast<float*>(p.o + (cell * (D / 4) + (d * 64 + tx * DW + e) / 4) * p.part_rows + r)[(tx * DW + e) % 4] = y;
                }
            if (tx == 0) {
                if (!whole) p.ml[cell * p.part_rows + r] = make_float2(m[i], l[i]);
                else if (a.lse) a.lse[row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
            }
        }
        if (tid == 0 && it.t0 == 0 && !it.whole()) p.cut[blockIdx.x] = {start.line, it.begin, it.row0, it.rows, h, owner(start.line, it.end() - 1, p.ctas)};
    }
}

// Rows of a tile: 16 where sequences have that few (a token or two of the group's heads), else 64.
int tile_rows(const PagedArgs& a) { return (int64_t)a.T * a.G <= 16 * (int64_t)a.N ? 16 : 64; }

template <typename IO, int D, int R> cudaError_t launch(const PagedArgs& a, cudaStream_t st)
{
    using L = F32<D, R>;
    constexpr int smem = sizeof(typename L::Smem);
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(paged_f32_kernel<IO, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    Plan p;
    lay_out(p, a, R, L::KEYS, CTAS);
    e = launch_dependent(paged_f32_kernel<IO, D, R>, CTAS, FT, smem, st, a, p);
    if (e == cudaSuccess) e = launch_join<IO, D>(a, p, st);
    return e;
}

template <typename IO, int D> cudaError_t launch_rows(const PagedArgs& a, cudaStream_t st)
{
    return tile_rows(a) == 16 ? launch<IO, D, 16>(a, st) : launch<IO, D, 64>(a, st);
}
template <typename IO> cudaError_t launch_io(const PagedArgs& a, cudaStream_t st)
{
    switch (a.D) {
    case 32: return launch_rows<IO, 32>(a, st);
    case 64: return launch_rows<IO, 64>(a, st);
    case 128: return launch_rows<IO, 128>(a, st);
    default: return launch_rows<IO, 256>(a, st);
    }
}

}  // namespace

size_t paged_f32_workspace_bytes(const PagedArgs& a)
{
    Plan p;
    return lay_out(p, a, tile_rows(a), a.D == 256 ? 32 : 64, CTAS);
}

cudaError_t launch_paged_f32(const PagedArgs& a, cudaStream_t st) { return launch_io<float>(a, st); }

}  // namespace kda
