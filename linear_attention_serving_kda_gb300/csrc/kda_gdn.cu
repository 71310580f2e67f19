// kda_gdn.cu -- the gated delta rule with one decay per head: the C entry
// points, the single-token form, and the row-by-row prefill of fp32 rows.
//
//     S = alpha S + k u^T,  u = beta (v - alpha S^T k),  o = scale S^T q
//
// The columns of S (dv) never meet, so any of them can be split over CTAs.
#include <cmath>
#include <cstring>

#include "kda_gdn.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

template <typename IO, int N> __device__ __forceinline__ void load_n(const IO* p, float (&x)[N])
{
    if constexpr (sizeof(IO) == 2 && N == 4) {
        const uint2 r = *reinterpret_cast<const uint2*>(p);
        x[0] = __uint_as_float(r.x << 16);
        x[1] = __uint_as_float(r.x & 0xffff0000u);
        x[2] = __uint_as_float(r.y << 16);
        x[3] = __uint_as_float(r.y & 0xffff0000u);
    } else if constexpr (sizeof(IO) == 4 && N == 4) {
        const float4 r = *reinterpret_cast<const float4*>(p);
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = ldv(p + i);
    }
}

// ------------------------------------------------------------ single token
//
// One CTA per (sequence, value head, tile of DVT columns).  The state is read
// once: with a = S^T k and b = S^T q of the OLD state in one sweep,
//     u = beta (v - alpha a),  o = scale (alpha b + (q.k) u),
// so the sweep's values wait in registers for u and go back as alpha S + k u^T.
// Bound: HBM, 8 bytes for each state value: 248 sequences of 32 heads of 128 x 128 165 us,
// 6.35 TB/s; one sequence 3.3 us, where the launch and two dependent loads are the bound.
constexpr int GD_WARPS = 8;

template <int DK, int DVT, typename IO, typename OUT>
__global__ void __launch_bounds__(GD_WARPS * 32) gdn_decode_kernel(const GdnArgs a, int dv)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int LPR = DVT / 4, RPP = 32 / LPR, RT = DK / (GD_WARPS * RPP), PER = DK / 32;
    static_assert(RT >= 1, "tile too narrow");
    __shared__ float ks[DK], qs[DK];
    __shared__ __align__(16) float red[GD_WARPS][2][DVT];
    const int tiles = dv / DVT;
    const int tile = blockIdx.x % tiles, u = blockIdx.x / tiles, h = u % a.Hv, seq = u / a.Hv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int row, end, slot;
    if (!gdn_unit(a, seq, row, end, slot)) return;
    const int hk = h / (a.Hv / a.Hk);
    const int col = tile * DVT + (lane % LPR) * 4;
    float* S = a.state + ((size_t)slot * a.Hv + h) * DK * dv + col;

    float4 s[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        s[r] = ld_stream4(S + (size_t)((r * GD_WARPS + warp) * RPP + lane / LPR) * dv);
    float q[PER], k[PER], v[4];
    load_n<IO, PER>(static_cast<const IO*>(a.q) + row * a.qs + hk * DK + lane * PER, q);
    load_n<IO, PER>(static_cast<const IO*>(a.k) + row * a.ks + hk * DK + lane * PER, k);
    load_n<IO, 4>(static_cast<const IO*>(a.v) + row * a.vs + h * dv + col, v);
    const size_t gi = (size_t)row * a.Hv + h;
    const float alpha = expf(gdn_log_alpha(expf(a.A_log[h]), ldv(static_cast<const IO*>(a.a) + gi), a.dt_bias[h]));
    const float beta = sigmoidf_(ldv(static_cast<const IO*>(a.b) + gi));
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        qq = fmaf(q[i], q[i], qq);
        kk = fmaf(k[i], k[i], kk);
        qk = fmaf(q[i], k[i], qk);
    }
    qq = warp_sum(qq);
    kk = warp_sum(kk);
    qk = warp_sum(qk);
    if (a.l2) {
        const float rq = rsqrtf(qq + a.l2_eps), rk = rsqrtf(kk + a.l2_eps);
        qk *= rq * rk;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            q[i] *= rq;
            k[i] *= rk;
        }
    }
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            qs[lane * PER + i] = q[i];
            ks[lane * PER + i] = k[i];
        }
    }
    __syncthreads();
    float da[4] = {}, db[4] = {};
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = (r * GD_WARPS + warp) * RPP + lane / LPR;
        const float ki = ks[i], qi = qs[i];
        const float x[4] = {s[r].x, s[r].y, s[r].z, s[r].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            da[c] = fmaf(ki, x[c], da[c]);
            db[c] = fmaf(qi, x[c], db[c]);
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            da[c] += __shfl_xor_sync(0xffffffffu, da[c], o);
            db[c] += __shfl_xor_sync(0xffffffffu, db[c], o);
        }
    if (lane < LPR) {
        *reinterpret_cast<float4*>(&red[warp][0][lane * 4]) = make_float4(da[0], da[1], da[2], da[3]);
        *reinterpret_cast<float4*>(&red[warp][1][lane * 4]) = make_float4(db[0], db[1], db[2], db[3]);
    }
    __syncthreads();
    float sa[4] = {}, sb[4] = {}, uu[4];
#pragma unroll
    for (int w = 0; w < GD_WARPS; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&red[w][0][(lane % LPR) * 4]);
        sa[0] += x.x; sa[1] += x.y; sa[2] += x.z; sa[3] += x.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) uu[c] = beta * (v[c] - alpha * sa[c]);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = (r * GD_WARPS + warp) * RPP + lane / LPR;
        const float ki = ks[i];
        float4 n;
        n.x = fmaf(ki, uu[0], alpha * s[r].x);
        n.y = fmaf(ki, uu[1], alpha * s[r].y);
        n.z = fmaf(ki, uu[2], alpha * s[r].z);
        n.w = fmaf(ki, uu[3], alpha * s[r].w);
        st_stream4(S + (size_t)i * dv, n);
    }
    if (warp == 0 && lane < LPR) {
#pragma unroll
        for (int w = 0; w < GD_WARPS; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&red[w][1][lane * 4]);
            sb[0] += x.x; sb[1] += x.y; sb[2] += x.z; sb[3] += x.w;
        }
        OUT* o = static_cast<OUT*>(a.out) + gi * dv + col;
#pragma unroll
        for (int c = 0; c < 4; ++c) stv(o + c, a.scale * fmaf(qk, uu[c], alpha * sb[c]));
    }
}

template <int DK, typename IO, typename OUT> cudaError_t decode_dk(const GdnArgs& a, int dv, cudaStream_t st)
{
    // Narrower tiles while there is less than one CTA for every SM (32 heads of 128: 3.3 us with
    // 32 columns a CTA, 5.3 with 128; 250 times as many 183 us with 32, 165 with 128).
    int t = dv;
    while (t > 32 && (long long)a.N * a.Hv * (dv / t) < sm_count()) t /= 2;
    const unsigned g = (unsigned)((long long)a.N * a.Hv * (dv / t));
    if (t == 128) return launch_dependent(gdn_decode_kernel<DK, 128, IO, OUT>, g, GD_WARPS * 32, 0, st, a, dv);
    if (t == 64) return launch_dependent(gdn_decode_kernel<DK, 64, IO, OUT>, g, GD_WARPS * 32, 0, st, a, dv);
    return launch_dependent(gdn_decode_kernel<DK, 32, IO, OUT>, g, GD_WARPS * 32, 0, st, a, dv);
}

template <typename IO, typename OUT> cudaError_t decode_io(const GdnArgs& a, int dk, int dv, cudaStream_t st)
{
    if (dk == 128) return decode_dk<128, IO, OUT>(a, dv, st);
    if (dk == 64) return decode_dk<64, IO, OUT>(a, dv, st);
    return decode_dk<32, IO, OUT>(a, dv, st);
}

// ------------------------------------------------------------ fp32 rows, one by one
//
// One CTA per (sequence, value head, 32 columns), the state in registers:
// lane (part, column) of a warp holds a quarter of a column.  Rows are staged
// sixteen at a time.  Bound: the chain of rows (two dot products across four
// lanes each), not bandwidth: ROWS_NOTE.
constexpr int GR_WARPS = 4, GR_COLS = 32, GR_ROWS = 16;

template <int DK> __global__ void __launch_bounds__(GR_WARPS * 32) gdn_rows_kernel(const GdnArgs a, int dv)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int PER = DK / 32, M = DK / 16, RW = GR_ROWS / GR_WARPS;
    __shared__ __align__(16) float qs[GR_ROWS][DK], ks[GR_ROWS][DK], vs[GR_ROWS][GR_COLS];
    __shared__ float al[GR_ROWS], be[GR_ROWS];
    const int tiles = dv / GR_COLS;
    const int tile = blockIdx.x % tiles, u = blockIdx.x / tiles, h = u % a.Hv, seq = u / a.Hv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = lane >> 3, c = warp * 8 + (lane & 7);
    int begin, end, slot;
    if (!gdn_unit(a, seq, begin, end, slot)) return;
    const int hk = h / (a.Hv / a.Hk);
    float* S = a.state + ((size_t)slot * a.Hv + h) * DK * dv + tile * GR_COLS + c;
    // the lane's rows of the state: 16 m + 4 part + 0..3
    float s[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[m][j] = S[(size_t)(16 * m + 4 * part + j) * dv];
    const float* q = static_cast<const float*>(a.q) + hk * DK + lane * PER;
    const float* k = static_cast<const float*>(a.k) + hk * DK + lane * PER;
    const float* v = static_cast<const float*>(a.v) + h * dv + tile * GR_COLS;
    float* out = static_cast<float*>(a.out) + (size_t)h * dv + tile * GR_COLS + c;
    const float ea = expf(a.A_log[h]), dt = a.dt_bias[h];

    for (int r0 = begin; r0 < end; r0 += GR_ROWS) {
        const int n = min(GR_ROWS, end - r0);
        float qr[RW][PER], kr[RW][PER];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = warp * RW + i;
            if (r < n) {
                load_n<float, PER>(q + (long long)(r0 + r) * a.qs, qr[i]);
                load_n<float, PER>(k + (long long)(r0 + r) * a.ks, kr[i]);
            }
        }
        __syncthreads();  // the rows staged before are done with
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = warp * RW + i;
            if (r >= n) continue;
            float rq = 1.f, rk = 1.f;
            if (a.l2) {
                float qq = 0.f, kk = 0.f;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    qq = fmaf(qr[i][j], qr[i][j], qq);
                    kk = fmaf(kr[i][j], kr[i][j], kk);
                }
                rq = rsqrtf(warp_sum(qq) + a.l2_eps);
                rk = rsqrtf(warp_sum(kk) + a.l2_eps);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                qs[r][lane * PER + j] = qr[i][j] * rq;
                ks[r][lane * PER + j] = kr[i][j] * rk;
            }
        }
        for (int i = tid; i < n * GR_COLS; i += GR_WARPS * 32)
            vs[i / GR_COLS][i % GR_COLS] = v[(long long)(r0 + i / GR_COLS) * a.vs + i % GR_COLS];
        if (tid < n) {
            const size_t gi = (size_t)(r0 + tid) * a.Hv + h;
            al[tid] = expf(gdn_log_alpha(ea, static_cast<const float*>(a.a)[gi], dt));
            be[tid] = sigmoidf_(static_cast<const float*>(a.b)[gi]);
        }
        __syncthreads();
        for (int r = 0; r < n; ++r) {
            const float alpha = al[r];
            float d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 kv = *reinterpret_cast<const float4*>(&ks[r][16 * m + 4 * part]);
                s[m][0] *= alpha; s[m][1] *= alpha; s[m][2] *= alpha; s[m][3] *= alpha;
                d0 = fmaf(kv.x, s[m][0], d0);
                d1 = fmaf(kv.y, s[m][1], d1);
                d0 = fmaf(kv.z, s[m][2], d0);
                d1 = fmaf(kv.w, s[m][3], d1);
            }
            float d = d0 + d1;
            d += __shfl_xor_sync(0xffffffffu, d, 8);
            d += __shfl_xor_sync(0xffffffffu, d, 16);
            const float uu = be[r] * (vs[r][c] - d);
            d0 = d1 = 0.f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 kv = *reinterpret_cast<const float4*>(&ks[r][16 * m + 4 * part]);
                const float4 qv = *reinterpret_cast<const float4*>(&qs[r][16 * m + 4 * part]);
                s[m][0] = fmaf(kv.x, uu, s[m][0]);
                s[m][1] = fmaf(kv.y, uu, s[m][1]);
                s[m][2] = fmaf(kv.z, uu, s[m][2]);
                s[m][3] = fmaf(kv.w, uu, s[m][3]);
                d0 = fmaf(qv.x, s[m][0], d0);
                d1 = fmaf(qv.y, s[m][1], d1);
                d0 = fmaf(qv.z, s[m][2], d0);
                d1 = fmaf(qv.w, s[m][3], d1);
            }
            float o = d0 + d1;
            o += __shfl_xor_sync(0xffffffffu, o, 8);
            o += __shfl_xor_sync(0xffffffffu, o, 16);
            if (part == 0) out[(size_t)(r0 + r) * a.Hv * dv] = a.scale * o;
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[(size_t)(16 * m + 4 * part + j) * dv] = s[m][j];
}

// ------------------------------------------------------------ checks

int check_gdn(const kda_gdn_params* p)
{
    if (!p) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_heads_k <= 0 || p->num_heads_v <= 0 || p->num_heads_v > 1024 || p->num_heads_v % p->num_heads_k != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    for (int d : {p->head_dim_k, p->head_dim_v})
        if (!(d == 32 || d == 64 || d == 128)) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (p->l2_norm != 0 && p->l2_norm != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (p->l2_norm && !(std::isfinite(p->l2_eps) && p->l2_eps >= 0.0f)) return KDA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(p->scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (!known_dtype(p->io_dtype) || !known_dtype(p->out_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (p->io_dtype == KDA_DTYPE_F32 && p->out_dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_slots <= 0) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t unit = 16 / io_size(p->io_dtype);
    const int64_t dense[3] = {(int64_t)p->num_heads_k * p->head_dim_k, (int64_t)p->num_heads_k * p->head_dim_k,
                              (int64_t)p->num_heads_v * p->head_dim_v};
    const int64_t given[3] = {p->q_row_stride, p->k_row_stride, p->v_row_stride};
    for (int i = 0; i < 3; ++i)
        if (given[i] != 0 && (given[i] < dense[i] || given[i] % unit != 0 || given[i] > ((int64_t)1 << 28)))
            return KDA_ERR_INVALID_ARGUMENT;
    return check_ptrs({p->A_log, p->dt_bias});
}

void fill_gdn(GdnArgs& g, const kda_gdn_params* p)
{
    std::memset(&g, 0, sizeof(g));
    g.Hk = p->num_heads_k;
    g.Hv = p->num_heads_v;
    g.num_slots = p->num_slots;
    g.l2 = p->l2_norm;
    g.l2_eps = p->l2_eps;
    g.scale = p->scale;
    g.A_log = p->A_log;
    g.dt_bias = p->dt_bias;
    g.qs = p->q_row_stride ? p->q_row_stride : (long long)p->num_heads_k * p->head_dim_k;
    g.ks = p->k_row_stride ? p->k_row_stride : (long long)p->num_heads_k * p->head_dim_k;
    g.vs = p->v_row_stride ? p->v_row_stride : (long long)p->num_heads_v * p->head_dim_v;
}

// Pointers of a call over `rows` rows of N sequences; `out`, the states and
// the workspace (`need` bytes of it) overlap no input and not each other.
int check_rows(const kda_gdn_params* p, const GdnArgs& g, int64_t rows, int64_t N, const int32_t* cu_seqlens, const void* q,
               const void* k, const void* v, const void* gate, const void* beta, const int32_t* slots,
               const float* rec_state, const void* out, const void* workspace, size_t need)
{
    int rc;
    if ((rc = check_ptrs({q, k, v, gate, beta, rec_state, out})) != KDA_OK || (rc = check_opt(slots)) != KDA_OK)
        return rc;
    const size_t io = io_size(p->io_dtype), kw = (size_t)p->num_heads_k * p->head_dim_k,
                 vw = (size_t)p->num_heads_v * p->head_dim_v;
    const size_t nout = (size_t)rows * vw * io_size(p->out_dtype);
    const size_t nstate = (size_t)p->num_slots * vw * p->head_dim_k * sizeof(float);
    const size_t heads = (size_t)p->num_heads_v * sizeof(float);
    const void* in[9] = {q, k, v, gate, beta, cu_seqlens, slots, p->A_log, p->dt_bias};
    const size_t size[9] = {((rows - 1) * g.qs + kw) * io, ((rows - 1) * g.ks + kw) * io, ((rows - 1) * g.vs + vw) * io,
                            (size_t)rows * p->num_heads_v * io, (size_t)rows * p->num_heads_v * io,
                            (size_t)(N + 1) * sizeof(int32_t), (size_t)N * sizeof(int32_t), heads, heads};
    for (int i = 0; i < 9; ++i)
        if (overlap(out, nout, in[i], size[i]) || overlap(rec_state, nstate, in[i], size[i]) ||
            overlap(workspace, need, in[i], size[i]))
            return KDA_ERR_INVALID_ARGUMENT;
    return overlap(out, nout, rec_state, nstate) || overlap(workspace, need, out, nout) ||
                   overlap(workspace, need, rec_state, nstate) ? KDA_ERR_INVALID_ARGUMENT : KDA_OK;
}

}  // namespace

cudaError_t launch_gdn_rows(const GdnArgs& a, int dk, int dv, cudaStream_t st)
{
    const unsigned g = (unsigned)((long long)a.N * a.Hv * (dv / GR_COLS));
    if (dk == 128) return launch_dependent(gdn_rows_kernel<128>, g, GR_WARPS * 32, 0, st, a, dv);
    if (dk == 64) return launch_dependent(gdn_rows_kernel<64>, g, GR_WARPS * 32, 0, st, a, dv);
    return launch_dependent(gdn_rows_kernel<32>, g, GR_WARPS * 32, 0, st, a, dv);
}

}  // namespace kda

using namespace kda;

extern "C" {

KDA_API size_t kda_gdn_prefill_workspace_bytes(const kda_gdn_params* p, int32_t N, int32_t T)
{
    if (check_gdn(p) != KDA_OK || N <= 0 || T <= 0 || p->io_dtype != KDA_DTYPE_BF16) return 0;
    return gdn_chunk_workspace_bytes(p->num_heads_k, p->num_heads_v, p->head_dim_k, p->out_dtype == KDA_DTYPE_BF16, N, T);
}

KDA_API int kda_gdn_prefill_varlen(const kda_gdn_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T,
                                   const void* q, const void* k, const void* v, const void* gate, const void* beta,
                                   const int32_t* slots, float* rec_state, void* out, void* workspace,
                                   size_t ws_bytes, int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_gdn(p);
    if (rc != KDA_OK) return rc;
    if (N < 0 || T < 0 || ((int64_t)T / 64 + 4 * (int64_t)N) * p->num_heads_v > INT32_MAX) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0 || T == 0) return KDA_OK;
    GdnArgs g;
    fill_gdn(g, p);
    if ((rc = check_ptrs({cu_seqlens})) != KDA_OK) return rc;
    const size_t need = kda_gdn_prefill_workspace_bytes(p, N, T);
    if ((rc = check_rows(p, g, T, N, cu_seqlens, q, k, v, gate, beta, slots, rec_state, out, workspace, need)) != KDA_OK) return rc;
    if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return KDA_ERR_WORKSPACE;
    if ((rc = check_device()) != KDA_OK) return rc;
    g.N = N;
    g.T = T;
    g.cu_seqlens = cu_seqlens;
    g.q = q; g.k = k; g.v = v; g.a = gate; g.b = beta;
    g.slots = slots;
    g.state = rec_state;
    g.out = out;
    g.workspace = workspace;
    g.dev_status = dev_status;
    const cudaError_t e = p->io_dtype == KDA_DTYPE_BF16
                              ? launch_gdn_chunk(g, p->head_dim_k, p->head_dim_v, p->out_dtype == KDA_DTYPE_BF16, stream)
                              : launch_gdn_rows(g, p->head_dim_k, p->head_dim_v, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

KDA_API int kda_gdn_decode(const kda_gdn_params* p, int32_t B, const void* q, const void* k, const void* v,
                           const void* gate, const void* beta, const int32_t* slots, float* rec_state, void* out,
                           int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_gdn(p);
    if (rc != KDA_OK) return rc;
    if (B < 0 || (int64_t)B * p->num_heads_v * 4 > INT32_MAX) return KDA_ERR_INVALID_ARGUMENT;
    if (B == 0) return KDA_OK;
    GdnArgs g;
    fill_gdn(g, p);
    if ((rc = check_rows(p, g, B, B, nullptr, q, k, v, gate, beta, slots, rec_state, out, nullptr, 0)) != KDA_OK) return rc;
    if ((rc = check_device()) != KDA_OK) return rc;
    g.N = g.T = B;
    g.q = q; g.k = k; g.v = v; g.a = gate; g.b = beta;
    g.slots = slots;
    g.state = rec_state;
    g.out = out;
    g.dev_status = dev_status;
    const int dk = p->head_dim_k, dv = p->head_dim_v;
    const cudaError_t e = p->io_dtype == KDA_DTYPE_F32    ? decode_io<float, float>(g, dk, dv, stream)
                          : p->out_dtype == KDA_DTYPE_BF16 ? decode_io<__nv_bfloat16, __nv_bfloat16>(g, dk, dv, stream)
                                                           : decode_io<__nv_bfloat16, float>(g, dk, dv, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // extern "C"
