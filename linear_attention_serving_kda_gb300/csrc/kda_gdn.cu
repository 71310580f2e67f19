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
// lane (columns, part) of a warp holds an eighth of two columns, so that a value of k or q
// from shared memory serves both (with a quarter of one column a lane those
// reads were the bound: 982 us where these take 660).  As for single
// tokens both of a row's dot products read the OLD state, so a row's
// dependent steps are one product, two shuffles and the update.  Rows are
// staged sixteen at a time, the next ones loaded meanwhile.  Bound: issue slots where
// there are many chains (packed arithmetic: two values an instruction), a row's steps where there
// are few, never bandwidth: 4096 rows of 8 sequences,
// 32 heads of 128 x 128, take 660 us, 2048 rows of one sequence 569 us.
constexpr int GR_WARPS = 4, GR_COLS = 32, GR_ROWS = 16;

template <int DK> __global__ void __launch_bounds__(GR_WARPS * 32) gdn_rows_kernel(const GdnArgs a, int dv)
{
    ptx::grid_dependency_wait();
    constexpr int PER = DK / 32, M = DK / 32, RW = GR_ROWS / GR_WARPS;
    __shared__ __align__(16) float qs[GR_ROWS][DK], ks[GR_ROWS][DK], vs[GR_ROWS][GR_COLS];
    __shared__ float al[GR_ROWS], be[GR_ROWS], qk[GR_ROWS];
    const int tiles = dv / GR_COLS;
    const int tile = blockIdx.x % tiles, u = blockIdx.x / tiles, h = u % a.Hv;
    __shared__ int found;
    const int seq = ranked_seq(a.cu_seqlens, a.N, u / a.Hv, &found);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = lane & 7, c0 = warp * 8 + (lane >> 3) * 2, odd = lane & 1;
    int begin, end, slot;
    if (!gdn_unit(a, seq, begin, end, slot)) return;
    const int hk = h / (a.Hv / a.Hk);
    float* S = a.state + ((size_t)slot * a.Hv + h) * DK * dv + tile * GR_COLS + c0;
    // of columns c0 and c0 + 1 the lane's rows of the state, 32 m + 4 part + 0..3, two by two
    float2 s[2][M][2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float* p = S + (size_t)(32 * m + 4 * part + 2 * j) * dv;
            const float2 x = *reinterpret_cast<const float2*>(p), y = *reinterpret_cast<const float2*>(p + dv);
            s[0][m][j] = make_float2(x.x, y.x);
            s[1][m][j] = make_float2(x.y, y.y);
        }
    const float* q = static_cast<const float*>(a.q) + hk * DK + lane * PER;
    const float* k = static_cast<const float*>(a.k) + hk * DK + lane * PER;
    const float* v = static_cast<const float*>(a.v) + h * dv + tile * GR_COLS + lane;
    float* out = static_cast<float*>(a.out) + (size_t)h * dv + tile * GR_COLS + c0 + odd;
    const float ea = expf(a.A_log[h]), dt = a.dt_bias[h];

    // rows warp * RW .. of a batch to a warp
    float qr[RW][PER], kr[RW][PER], vr[RW], gate = 0.f, beta = 0.f;
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = r0 + warp * RW + i;
            if (r < end) {
                load_n<float, PER>(q + (long long)r * a.qs, qr[i]);
                load_n<float, PER>(k + (long long)r * a.ks, kr[i]);
                vr[i] = v[(long long)r * a.vs];
            }
        }
        if (tid < GR_ROWS && r0 + tid < end) {
            gate = static_cast<const float*>(a.a)[(size_t)(r0 + tid) * a.Hv + h];
            beta = static_cast<const float*>(a.b)[(size_t)(r0 + tid) * a.Hv + h];
        }
    };
    fetch(begin);
    for (int r0 = begin; r0 < end; r0 += GR_ROWS) {
        const int n = min(GR_ROWS, end - r0);
        __syncthreads();  // the rows staged before are done with
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = warp * RW + i;
            if (r >= n) continue;
            float qq = 0.f, kk = 0.f, x = 0.f;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                qq = fmaf(qr[i][j], qr[i][j], qq);
                kk = fmaf(kr[i][j], kr[i][j], kk);
                x = fmaf(qr[i][j], kr[i][j], x);
            }
            float rq = 1.f, rk = 1.f;
            if (a.l2) {
                rq = rsqrtf(warp_sum(qq) + a.l2_eps);
                rk = rsqrtf(warp_sum(kk) + a.l2_eps);
            }
            x = warp_sum(x);
            if (lane == 0) qk[r] = x * rq * rk;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                qs[r][lane * PER + j] = qr[i][j] * rq;
                ks[r][lane * PER + j] = kr[i][j] * rk;
            }
            vs[r][lane] = vr[i];
        }
        if (tid < n) {
            al[tid] = expf(gdn_log_alpha(ea, gate, dt));
            be[tid] = sigmoidf_(beta);
        }
        __syncthreads();
        fetch(r0 + GR_ROWS);
        for (int r = 0; r < n; ++r) {
            const float alpha = al[r];
            float2 x[2], y[2], kp[M][2];  // k.S and q.S of both columns
#pragma unroll
            for (int e = 0; e < 2; ++e) x[e] = y[e] = both2(0.f);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 kv = *reinterpret_cast<const float4*>(&ks[r][32 * m + 4 * part]);
                const float4 qv = *reinterpret_cast<const float4*>(&qs[r][32 * m + 4 * part]);
                kp[m][0] = make_float2(kv.x, kv.y);
                kp[m][1] = make_float2(kv.z, kv.w);
                const float2 qp[2] = {make_float2(qv.x, qv.y), make_float2(qv.z, qv.w)};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[e] = fma2(kp[m][j], s[e][m][j], x[e]);
                        y[e] = fma2(qp[j], s[e][m][j], y[e]);
                    }
            }
            // over the eight parts: neighbours trade a column first, so that each lane ends with one column's sums
            const float2 d0 = make_float2(x[0].x + x[0].y, y[0].x + y[0].y), d1 = make_float2(x[1].x + x[1].y, y[1].x + y[1].y);
            const float2 mine = odd ? d1 : d0, other = odd ? d0 : d1;
            float2 d = add2(mine, make_float2(__shfl_xor_sync(0xffffffffu, other.x, 1), __shfl_xor_sync(0xffffffffu, other.y, 1)));
#pragma unroll
            for (int o = 2; o < 8; o <<= 1)
                d = add2(d, make_float2(__shfl_xor_sync(0xffffffffu, d.x, o), __shfl_xor_sync(0xffffffffu, d.y, o)));
            const float uu = be[r] * (vs[r][c0 + odd] - alpha * d.x), theirs = __shfl_xor_sync(0xffffffffu, uu, 1);
            const float2 u2[2] = {both2(odd ? theirs : uu), both2(odd ? uu : theirs)};
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[e][m][j] = fma2(kp[m][j], u2[e], mul2(both2(alpha), s[e][m][j]));
            if (part < 2) out[(size_t)(r0 + r) * a.Hv * dv] = a.scale * fmaf(qk[r], uu, alpha * d.y);
        }
    }
    ptx::grid_launch_dependents();  // not before: the next call's CTAs would crowd the SMs that are free
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float* p = S + (size_t)(32 * m + 4 * part + 2 * j) * dv;
            *reinterpret_cast<float2*>(p) = make_float2(s[0][m][j].x, s[1][m][j].x);
            *reinterpret_cast<float2*>(p + dv) = make_float2(s[0][m][j].y, s[1][m][j].y);
        }
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
    return gdn_chunk_workspace_bytes(p->num_heads_k, p->num_heads_v, p->head_dim_k, N, T);
}

KDA_API int kda_gdn_prefill_varlen(const kda_gdn_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T,
                                   const void* q, const void* k, const void* v, const void* gate, const void* beta,
                                   const int32_t* slots, float* rec_state, void* out, void* workspace,
                                   size_t ws_bytes, int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_gdn(p);
    if (rc != KDA_OK) return rc;
    if (N < 0 || T < 0 || T > KDA_MAX_ROWS || ((int64_t)T / 64 + 4 * (int64_t)N) * p->num_heads_v > INT32_MAX)
        return KDA_ERR_INVALID_ARGUMENT;
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
