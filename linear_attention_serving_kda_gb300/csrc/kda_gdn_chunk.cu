// kda_gdn_chunk.cu -- chunked prefill of the gated delta rule with one decay
// per head (bf16 rows), in chunks of C = 64 rows.
//
// With G the running sum of log alpha in the chunk, row by row:
//     A_rs = beta_r e^{G_r - G_s} k_r.k_s  (s < r),   T = (I + A)^-1
//     U    = T diag(beta) (V - diag(e^G) K S)
//     O    = diag(e^G) Q S + P U,   P_rs = e^{G_r - G_s} q_r.k_s  (s <= r)
//     S'   = e^{G_C} S + (diag(e^{G_C - G}) K)^T U
// All exponents are differences that are <= 0.
//
// A CTA owns one (sequence, value head, DVT columns of dv); nothing crosses
// columns, so these never meet.  Sixteen warps in four roles, a chunk apart:
//   - a loader: rows by tensor copies, and the raw products [K; Q] [K; Q]^T of
//     the next chunk as one tcgen05 product into TMEM (k.k, q.k and, on the
//     diagonal, both squared norms);
//   - eight prep warps, one row of [K; Q] a lane: the norms, P and A from
//     those, then T by forward substitution of the 16 x 16 diagonal blocks and
//     doubling; k and q rescaled in place;
//   - NW chain warps: each keeps S^T for 16 columns in registers as the
//     accumulator of a 16 x dk product and walks the chunks alone: S^T K^T,
//     R^T T^T (R = beta (V - ..)) and U^T K take their left operand straight
//     from the accumulators of the product before (the two fragment layouts
//     agree), so no chain warp ever waits for another one;
//   - an issuer and two output warps: Q S and P U as tcgen05 products of the
//     tiles that chain and prep leave, and the outputs' rows from TMEM.
//
// Precision: the state keeps fp32 accuracy.  One decay per head leaves k and q
// unscaled inside every product, so the rows' bf16 values are operands without
// loss: prep rescales each row by a power of two to a norm in [1, 2) and stores
// it as fp16 (exact down to 2^-17).  Every other operand that reaches the state
// is two fp16 values, high and low, about 22 bits: S and U and V - .. are scaled
// by a power of two per column so that the low part stays in fp16's range.  P
// and the outputs' reading of S and U keep the high part only where the
// outputs are bf16 (11 bits against their 8).
#include <cstddef>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kda_gdn.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int C = 64;
constexpr int THREADS = 512;
constexpr int PREP_WARP = 8, PREP = 256;  // first prep warp, prep threads
constexpr int XS = 20;                    // row stride of the fp32 diagonal blocks
// TMEM columns: two raw products of 128, Q S, P U
constexpr int TM_PROD = 0, TM_QS = 256, TM_PU = 320, TM_COLS = 512;

// ------------------------------------------------------------ fragments

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack_h(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
// x, y as high and low fp16 pairs
__device__ __forceinline__ void split_h(float x, float y, uint32_t& hi, uint32_t& lo)
{
    hi = pack_h(x, y);
    const float2 f = unpack_h(hi);
    lo = pack_h(x - f.x, y - f.y);
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Byte offsets of 16-byte piece `c` of row `r` in the tiles, all with 128-byte
// rows, pieces permuted within eight rows (as a tensor copy with the 128-byte
// swizzle leaves them and the tensor core's descriptors expect them), so that
// eight rows' same piece lie in distinct banks.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return (uint32_t)(r * 128 + (((c ^ r) & 7) << 4)); }
// [K; Q]: 128 rows, 64 values wide, one such tile after the other
__device__ __forceinline__ uint32_t kq_at(int r, int c) { return (uint32_t)((c >> 3) * 16384) + tile_at(r, c); }
// the same with ROWS rows
template <int ROWS> __device__ __forceinline__ uint32_t half_at(int r, int c)
{
    return (uint32_t)((c >> 3) * ROWS * 128) + tile_at(r, c);
}
// V: 64 rows of W values; 64-byte rows with the 64-byte swizzle where W = 32
template <int W> __device__ __forceinline__ uint32_t v_at(int r, int c)
{
    if constexpr (W == 64) return tile_at(r, c);
    else return (uint32_t)(r * 64 + ((c ^ (r >> 1)) & 3) * 16);
}

// 2^-e and 2^e for the e that brings m into [1, 2), kept within 2^+-60 (so
// that products of two such factors stay finite).
__device__ __forceinline__ void pow2_scale(float m, float& down, float& up)
{
    const uint32_t e = min(max((__float_as_uint(m) >> 23) & 255u, 67u), 187u);
    down = __uint_as_float((254u - e) << 23);
    up = __uint_as_float(e << 23);
}
// The same for sqrt(m), m >= 0.
__device__ __forceinline__ void pow2_scale_sqrt(float m, float& down, float& up)
{
    const int e = min(max((((int)(__float_as_uint(m) >> 23) & 255) + 1 - 128) >> 1, -60), 60);
    down = __uint_as_float((uint32_t)(127 - e) << 23);
    up = __uint_as_float((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ float exp2_sfu(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------ shared memory

template <int DK, int DVT, bool F32> struct Smem {
    static constexpr int PARTS = F32 ? 2 : 1;
    static constexpr int HALVES = DK <= 64 ? 1 : DK / 64;  // 64-wide tiles a row spans (dk = 32: half of one)
    unsigned char kq[3][HALVES * 16384];   // bf16 rows of k, then q; fp16 later
    unsigned char v[3][C * DVT * 2];
    // T high, P high, T low (and P low): 64 x 64 fp16 tiles; T over P is one 128-row operand
    unsigned char tp[2][(2 + PARTS) * 8192];
    unsigned char st[PARTS][HALVES * DVT * 128];  // S^T: a row a column of dv
    unsigned char ut[PARTS][DVT * 128];           // U^T likewise
    // read four at a time: each on a 16-byte boundary
    alignas(16) float x[C * XS];           // A's diagonal blocks, 16 x 16 each
    // per chunk row: beta; beta sk e^G; sk; e^{G_C - G}; scale sq e^G; scale sq
    float beta[2][C], ek[2][C], sk[2][C], w[2][C], e1[2][C], e2[2][C];
    alignas(16) float f1[2][DVT], f2[2][DVT];  // the scales of S^T's and U^T's columns
    alignas(16) float eg[C], gh[C], gl[C];  // e^G and G / ln 2 in two words
    alignas(16) float norm[2 * C];         // squared norms of k's and q's rows
    alignas(16) float row[2 * C], colk[C], down[2 * C];  // factors of A's and P's rows, of A's columns; of the stored rows
    float last[2];                         // e^{G_C}
    uint64_t loaded[3], kv_free[3];        // a chunk's rows; their last use
    uint64_t prod_full[2], prod_free[2];   // raw products
    uint64_t ready[2], tp_free[2];         // T, P and the factors; their last use
    uint64_t s_full, s_free, u_full[2];    // S^T's tile; U^T's
    uint64_t o_full, o_free;               // Q S and P U in TMEM (which frees U^T's tile); read
    uint32_t tmem;
    int found;

    __device__ __forceinline__ unsigned char* t_hi(int b) { return tp[b]; }
    __device__ __forceinline__ unsigned char* t_lo(int b) { return tp[b] + 16384; }
};

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, %0;" ::"n"(PREP) : "memory"); }
// the four warps that invert T
__device__ __forceinline__ void invert_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// Bounded waits: after one that gives up the others only look once, and the
// role reports it at its end.
struct Waiter {
    bool dead;
    __device__ __forceinline__ void operator()(uint64_t& bar, int phase)
    {
        if (!ptx::mbar_wait_short(&bar, phase & 1, dead ? 1u : 1u << 22)) dead = true;
    }
};

__device__ __forceinline__ void warp_arrive(uint64_t& bar, int lane)
{
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&bar);
}

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// ------------------------------------------------------------ prep

// (h, l) += (oh, ol) in double-word fp32
__device__ __forceinline__ void dw_add(float& h, float& l, float oh, float ol)
{
    const float s = __fadd_rn(h, oh), bb = __fsub_rn(s, h);
    const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(s, bb)), __fsub_rn(oh, bb));
    const float r = __fadd_rn(__fadd_rn(l, ol), e);
    h = __fadd_rn(s, r);
    l = __fsub_rn(r, __fsub_rn(h, s));
}

// One warp, rows 2 lane and 2 lane + 1 of a chunk: running sums of their log2
// decays g (double word: differences of large sums keep their small part).
template <class S> __device__ __forceinline__ void scan_rows(S& sm, int b, float2 g, int lane)
{
    float h = g.x, l = 0.f;
    dw_add(h, l, g.y, 0.f);
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const float oh = __shfl_up_sync(0xffffffffu, h, o), ol = __shfl_up_sync(0xffffffffu, l, o);
        if (lane >= o) dw_add(h, l, oh, ol);
    }
    const float th = __shfl_sync(0xffffffffu, h, 31), tl = __shfl_sync(0xffffffffu, l, 31);
    float ph = __shfl_up_sync(0xffffffffu, h, 1), pl = __shfl_up_sync(0xffffffffu, l, 1);
    if (lane == 0) ph = pl = 0.f;
    dw_add(ph, pl, g.x, 0.f);  // the lane's first row
    *reinterpret_cast<float2*>(&sm.gh[2 * lane]) = make_float2(ph, h);
    *reinterpret_cast<float2*>(&sm.gl[2 * lane]) = make_float2(pl, l);
    *reinterpret_cast<float2*>(&sm.eg[2 * lane]) = make_float2(exp2_sfu(ph + pl), exp2_sfu(h + l));
    *reinterpret_cast<float2*>(&sm.w[b][2 * lane]) =
        make_float2(exp2_sfu((th - ph) + (tl - pl)), exp2_sfu((th - h) + (tl - l)));
    if (lane == 0) sm.last[b] = exp2_sfu(th + tl);
}

// A row of [K; Q]: bf16 -> fp16 times a power of two, in place; zeros for a
// padded row (the copies took the next sequence's along).
template <int DK> __device__ __forceinline__ void convert_row(unsigned char* tile, int r, float down, bool real)
{
    const __nv_bfloat162 d = __float2bfloat162_rn(down);
#pragma unroll 1
    for (int c0 = 0; c0 < DK / 8; c0 += 4) {
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const uint4*>(tile + kq_at(r, c0 + c));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), d);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
                w[i] = real ? pack_h(bf_lo(u), bf_hi(u)) : 0u;
            }
            x[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(tile + kq_at(r, c0 + c)) = x[c];
    }
}

// x, y as fp16 high and low pairs at (r, s), (r, s + 1) of two operand tiles
__device__ __forceinline__ void put_pair(unsigned char* hi_tile, unsigned char* lo_tile, int r, int s, float x, float y)
{
    uint32_t hi, lo;
    split_h(x, y, hi, lo);
    const uint32_t o = tile_at(r, s >> 3) + (s & 7) * 2;
    *reinterpret_cast<uint32_t*>(hi_tile + o) = hi;
    *reinterpret_cast<uint32_t*>(lo_tile + o) = lo;
}

// Columns n0 .. n0 + 15, rows mt * 16 .. + 15 of  T21 = -T22 (A21 T11)  for the
// SIZE-blocks at (i0, j0): T11 and T22 are in the operand tiles, A21 in
// T21's place.
template <int SIZE> struct Merge {
    float pt[SIZE / 8][4];  // (A21 T11)^T, rows n: its accumulators are the next product's right operand
    template <class S> __device__ __forceinline__ void first(S& sm, int b, int i0, int j0, int n0, int lane)
    {
        const uint32_t th = ptx::smem_u32(sm.t_hi(b)), tl = ptx::smem_u32(sm.t_lo(b));
        const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
#pragma unroll
        for (int t = 0; t < SIZE / 8; ++t) pt[t][0] = pt[t][1] = pt[t][2] = pt[t][3] = 0.f;
#pragma unroll
        for (int kt = 0; kt < SIZE / 16; ++kt) {
            uint32_t ah[4], al[4], bh[SIZE / 16][4], bl[SIZE / 16][4];
            const uint32_t ao = tile_at(j0 + kt * 16 + brow, ((j0 + n0) >> 3) + bcol);
            ldsm_t(ah, th + ao);
            ldsm_t(al, tl + ao);
#pragma unroll
            for (int t = 0; t < SIZE / 16; ++t) {
                const uint32_t bo = tile_at(i0 + t * 16 + brow, ((j0 + kt * 16) >> 3) + bcol);
                ldsm(bh[t], th + bo);
                ldsm(bl[t], tl + bo);
            }
#pragma unroll
            for (int t = 0; t < SIZE / 8; ++t) mma(pt[t], ah, bh[t >> 1][2 * (t & 1)], bh[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
            for (int t = 0; t < SIZE / 8; ++t) mma(pt[t], ah, bl[t >> 1][2 * (t & 1)], bl[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
            for (int t = 0; t < SIZE / 8; ++t) mma(pt[t], al, bh[t >> 1][2 * (t & 1)], bh[t >> 1][2 * (t & 1) + 1]);
        }
    }
    template <class S> __device__ __forceinline__ void second(S& sm, int b, int i0, int mt, float (&o)[2][4], int lane)
    {
        const uint32_t th = ptx::smem_u32(sm.t_hi(b)), tl = ptx::smem_u32(sm.t_lo(b));
#pragma unroll
        for (int n = 0; n < 2; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
        for (int kt = 0; kt < SIZE / 16; ++kt) {
            uint32_t ah[4], al[4], bh[2][2], bl[2][2];
            const uint32_t ao = tile_at(i0 + mt * 16 + (lane & 15), ((i0 + kt * 16) >> 3) + (lane >> 4));
            ldsm(ah, th + ao);
            ldsm(al, tl + ao);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) split_h(pt[2 * kt + i][2 * n], pt[2 * kt + i][2 * n + 1], bh[n][i], bl[n][i]);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma(o[n], ah, bh[n][0], bh[n][1]);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma(o[n], ah, bl[n][0], bl[n][1]);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma(o[n], al, bh[n][0], bh[n][1]);
        }
    }
    template <class S>
    __device__ __forceinline__ void store(S& sm, int b, int i0, int j0, int n0, int mt, const float (&o)[2][4], int lane)
    {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                put_pair(sm.t_hi(b), sm.t_lo(b), i0 + mt * 16 + (lane >> 2) + i * 8, j0 + n0 + n * 8 + (lane & 3) * 2,
                         -o[n][2 * i], -o[n][2 * i + 1]);
    }
};

// Chunk m of prep warp w (n rows of it are real).  Lane and w & 3 give the
// row of [K; Q] whose products the warp reads, w >> 2 which half of k's rows it
// reads them against; the halves above the diagonal (w = 4 and 6) are left out.
// The loops stay rolled: this runs once a chunk beside the other roles' code,
// and what the instruction cache does not hold is fetched anew each time (at
// 150 KB of code that was the kernel's first stall).
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void prep_chunk(S& sm, int m, const GdnArgs& a, int n, float2 g, float2 beta, Waiter& wait,
                                           uint32_t tmem, int w, int lane)
{
    const int b = m & 1, slot = m % 3;
    const int lr = (w & 3) * 32 + lane, r = lr & (C - 1), type = lr >> 6, s0 = (w >> 2) * 32;  // type 0: k, 1: q
    const uint32_t at = tmem + ((uint32_t)((w & 3) * 32) << 16) + TM_PROD + b * 128;
    if (m >= 2) wait(sm.tp_free[b], (m - 2) >> 1);
    if (w == 4) {
        *reinterpret_cast<float2*>(&sm.beta[b][2 * lane]) = beta;
        scan_rows(sm, b, g, lane);
    } else {
        wait(sm.prod_full[b], m >> 1);
        ptx::tc_fence_after();
        if (w == 0 || w >= 5) {
            // the squared norms of 32 rows of k (w = 0, 5) or q: the diagonal
            const int c0 = w == 0 ? 0 : (w - 4) * 32;
            float y = 0.f;
#pragma unroll 1
            for (int c = 0; c < 32; c += 8) {
                float d[8];
                ptx::tmem_ld8(at + c0 + c, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) y = c + i == lane ? d[i] : y;
            }
            sm.norm[lr] = y;
        }
    }
    prep_sync();
    if (w < 4) {
        const float ss = sm.norm[lr];
        float down, up;
        pow2_scale_sqrt(ss, down, up);
        // the factor that makes the stored row the (normalised) row; none for a padded one
        const float nrm = r < n ? (a.l2 ? rsqrtf(ss + a.l2_eps) : 1.f) : 0.f, f = nrm * up;
        sm.down[lr] = down;
        if (type == 0) {
            const float be = sm.beta[b][r];
            sm.sk[b][r] = f;
            sm.ek[b][r] = be * f * sm.eg[r];
            sm.colk[r] = nrm;  // A comes from the raw rows' products
            sm.row[r] = be * nrm;
        } else {
            sm.e1[b][r] = a.scale * f * sm.eg[r];
            sm.e2[b][r] = a.scale * f;
            sm.row[lr] = down;  // P is that of the stored rows
        }
    }
    prep_sync();
    if (w != 4 && w != 6) {
        // the lane's row of A (beta_r |..| e^{G_r - G_s} k_r.k_s) or P, zero from the diagonal (or past it) on
        const float rh = sm.gh[r], rl = sm.gl[r], rf = sm.row[lr];
        const float* cf = type == 0 ? sm.colk : sm.down;
        const int lim = r < n ? r + type : 0;
        unsigned char* hi_tile = sm.tp[b];
        unsigned char* lo_tile = sm.tp[b] + 16384;
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {
            uint32_t hi[4], lo[4];
            float v[8], d[8];
            ptx::tmem_ld8(at + s0 + p * 8, d);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int s = s0 + p * 8 + z * 4;
                const float4 ch = *reinterpret_cast<const float4*>(&sm.gh[s]);
                const float4 cl = *reinterpret_cast<const float4*>(&sm.gl[s]);
                const float4 c4 = *reinterpret_cast<const float4*>(&cf[s]);
                const float h4[4] = {ch.x, ch.y, ch.z, ch.w}, l4[4] = {cl.x, cl.y, cl.z, cl.w}, f4[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = exp2_sfu((rh - h4[i]) + (rl - l4[i]));
                    v[z * 4 + i] = s + i < lim ? (rf * f4[i]) * e * d[z * 4 + i] : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) split_h(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
            const int c = (s0 >> 3) + p;
            *reinterpret_cast<uint4*>(hi_tile + tile_at(lr, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (F32 || type == 0) *reinterpret_cast<uint4*>(lo_tile + tile_at(lr, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (type == 0 && (r >> 4) == (c >> 1)) {
                float* x = &sm.x[r * XS + (c & 1) * 8];
                *reinterpret_cast<float4*>(x) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(x + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }
    ptx::tc_fence_before();
    warp_arrive(sm.prod_free[b], lane);
    prep_sync();
    if (w >= 4) {
        // meanwhile the rows themselves
        const int row = (w - 4) * 32 + lane, rr = row & (C - 1);
        wait(sm.loaded[slot], m / 3);
        convert_row<DK>(sm.kq[slot], row, sm.down[row], rr < n);
        if (row < C && rr >= n)
#pragma unroll 1
            for (int c = 0; c < DVT / 8; ++c)
                *reinterpret_cast<uint4*>(sm.v[slot] + v_at<DVT>(rr, c)) = make_uint4(0, 0, 0, 0);
    } else {
        {
            // a diagonal block a warp: forward substitution, a column a lane (both
            // halves of the warp: one stores the high parts, one the low)
            const int d0 = w * 16, c = lane & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float acc = i == c ? 1.f : 0.f, acc2 = 0.f;
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&sm.x[(d0 + i) * XS + j]);
                    acc = fmaf(-f.x, x[j], acc);
                    if (j + 1 < i) acc2 = fmaf(-f.y, x[j + 1], acc2);
                    if (j + 2 < i) acc = fmaf(-f.z, x[j + 2], acc);
                    if (j + 3 < i) acc2 = fmaf(-f.w, x[j + 3], acc2);
                }
                x[i] = acc + acc2;
            }
            unsigned char* tile = lane < 16 ? sm.t_hi(b) : sm.t_lo(b);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const __half hi = __float2half_rn(x[i]);
                const __half lo = __float2half_rn(x[i] - __half2float(hi));
                *reinterpret_cast<__half*>(tile + tile_at(d0 + i, (d0 + c) >> 3) + (c & 7) * 2) = lane < 16 ? hi : lo;
            }
        }
        invert_sync();
        float o[2][4];
        if (w < 2) {
            const int j0 = w * 32, i0 = j0 + 16;
            Merge<16> mg;
            mg.first(sm, b, i0, j0, 0, lane);
            mg.second(sm, b, i0, 0, o, lane);
            __syncwarp();
            mg.store(sm, b, i0, j0, 0, 0, o, lane);
        }
        invert_sync();
        Merge<32> mg;
        const int n0 = (w & 1) * 16, mt = w >> 1;
        mg.first(sm, b, 32, 0, n0, lane);
        mg.second(sm, b, 32, mt, o, lane);
        invert_sync();  // every warp has read A21
        mg.store(sm, b, 32, 0, n0, mt, o, lane);
    }
    ptx::fence_proxy_async_smem();
    warp_arrive(sm.ready[b], lane);
}

// ------------------------------------------------------------ chain

// Chunk m of a chain warp: 16 columns of dv.  s holds S^T times g[0] (column
// lane / 4) and g[1] (eight further), ig their inverses.
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void chain_chunk(S& sm, int m, float (&s)[DK / 8][4], float (&ig)[2], Waiter& wait, int warp,
                                            int lane)
{
    const int slot = m % 3, b = m & 1, q2 = (lane & 3) * 2;
    const uint32_t kb = ptx::smem_u32(sm.kq[slot]), vb = ptx::smem_u32(sm.v[slot]);
    const uint32_t tb[2] = {ptx::smem_u32(sm.t_hi(b)), ptx::smem_u32(sm.t_lo(b))};
    const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;  // K-contiguous operand
    const int trow = lane & 15, tcol = lane >> 4;                                 // transposed operand
    if (m > 0) wait(sm.s_free, m - 1);

    // S^T K^T, each k-tile's fragments made a tile ahead
    float r[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[t][i] = 0.f;
    __half2 m0 = __float2half2_rn(0.f), m1 = m0;
    uint32_t f[2][4][4], hi[2][4], lo[2][4];
    auto left = [&](int kt) {  // k-tile kt of S^T, split, also for the outputs
#pragma unroll
        for (int t = 0; t < 4; ++t) ldsm(f[kt & 1][t], kb + kq_at(t * 16 + brow, kt * 2 + bcol));
        uint32_t(&x)[4] = hi[kt & 1], (&y)[4] = lo[kt & 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* v = &s[2 * kt + (i >> 1)][2 * (i & 1)];
            split_h(v[0], v[1], x[i], y[i]);
            const __half2 h = __habs2(*reinterpret_cast<const __half2*>(&x[i]));
            if (i & 1) m1 = __hmax2(m1, h);
            else m0 = __hmax2(m0, h);
        }
        const uint32_t o = half_at<DVT>(warp * 16 + trow, kt * 2 + tcol);
        stsm(ptx::smem_u32(sm.st[0]) + o, x);
        if (F32) stsm(ptx::smem_u32(sm.st[F32 ? 1 : 0]) + o, y);
    };
    left(0);
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        if (kt + 1 < DK / 16) left(kt + 1);
        uint32_t(&e)[4][4] = f[kt & 1];
#pragma unroll
        for (int t = 0; t < 8; ++t) mma(r[t], hi[kt & 1], e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 8; ++t) mma(r[t], lo[kt & 1], e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
    }
    ptx::fence_proxy_async_smem();
    warp_arrive(sm.s_full, lane);
    // beta (V - e^G k.S), and each column's largest value
    float mr[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
        uint32_t v[4];  // V^T: rows t*8.. of columns gq, gq+8; then the next eight rows
        ldsm_t(v, vb + v_at<DVT>(t * 8 + brow, warp * 2 + bcol));
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float2 be = *reinterpret_cast<const float2*>(&sm.beta[b][(t + z) * 8 + q2]);
            const float2 ek = *reinterpret_cast<const float2*>(&sm.ek[b][(t + z) * 8 + q2]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float* x = &r[t + z][2 * i];
                x[0] = fmaf(-ek.x, x[0] * ig[i], be.x * bf_lo(v[2 * z + i]));
                x[1] = fmaf(-ek.y, x[1] * ig[i], be.y * bf_hi(v[2 * z + i]));
                mr[i] = fmaxf(mr[i], fmaxf(fabsf(x[0]), fabsf(x[1])));
            }
        }
    }
    float rd[2], ru[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) pow2_scale(quad_max(mr[i]), rd[i], ru[i]);
    // U^T = R^T T^T (T is lower triangular: k-tile kt meets rows from 16 kt on)
    float u[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[t][i] = 0.f;
    uint32_t f2[2][4][4];
    auto part = [&](int kt) {
#pragma unroll
        for (int t = kt; t < 4; ++t) {
            ldsm(f[kt & 1][t], tb[0] + tile_at(t * 16 + brow, kt * 2 + bcol));
            ldsm(f2[kt & 1][t], tb[1] + tile_at(t * 16 + brow, kt * 2 + bcol));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = &r[2 * kt + (i >> 1)][2 * (i & 1)];
            split_h(x[0] * rd[i & 1], x[1] * rd[i & 1], hi[kt & 1][i], lo[kt & 1][i]);
        }
    };
    part(0);
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        if (kt + 1 < 4) part(kt + 1);
        uint32_t(&th)[4][4] = f[kt & 1], (&tl)[4][4] = f2[kt & 1], (&x)[4] = hi[kt & 1], (&y)[4] = lo[kt & 1];
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], x, th[t >> 1][2 * (t & 1)], th[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], y, th[t >> 1][2 * (t & 1)], th[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], x, tl[t >> 1][2 * (t & 1)], tl[t >> 1][2 * (t & 1) + 1]);
    }
    // times k's row factor; the largest values with and without the decay to the chunk's end
    float mu[2] = {0.f, 0.f}, mw[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float2 sk = *reinterpret_cast<const float2*>(&sm.sk[b][t * 8 + q2]);
        const float2 w = *reinterpret_cast<const float2*>(&sm.w[b][t * 8 + q2]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float* x = &u[t][2 * i];
            x[0] *= sk.x * ru[i];
            x[1] *= sk.y * ru[i];
            mu[i] = fmaxf(mu[i], fmaxf(fabsf(x[0]), fabsf(x[1])));
            mw[i] = fmaxf(mw[i], fmaxf(fabsf(x[0]) * w.x, fabsf(x[1]) * w.y));
        }
    }
    const float last = sm.last[b];
    float ud[2], dec[2], g[2];
    {
        const float ms[2] = {fmaxf(__low2float(m0), __high2float(m0)) * ig[0],
                             fmaxf(__low2float(m1), __high2float(m1)) * ig[1]};
        const float old[2] = {ig[0], ig[1]};
        float up[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pow2_scale(quad_max(mu[i]), ud[i], up[i]);
            pow2_scale(quad_max(fmaxf(mw[i], ms[i] * last)), g[i], ig[i]);
            dec[i] = last * (g[i] * old[i]);
        }
        if (m > 0) wait(sm.o_full, m - 1);
        if ((lane & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sm.f1[b][warp * 16 + (lane >> 2) + i * 8] = old[i];
                sm.f2[b][warp * 16 + (lane >> 2) + i * 8] = up[i];
            }
        }
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* v = &u[2 * kt + (i >> 1)][2 * (i & 1)];
            if (F32) split_h(v[0] * ud[i & 1], v[1] * ud[i & 1], x[i], y[i]);
            else x[i] = pack_h(v[0] * ud[i & 1], v[1] * ud[i & 1]);
        }
        const uint32_t o = half_at<DVT>(warp * 16 + trow, kt * 2 + tcol);
        stsm(ptx::smem_u32(sm.ut[0]) + o, x);
        if (F32) stsm(ptx::smem_u32(sm.ut[F32 ? 1 : 0]) + o, y);
    }
    ptx::fence_proxy_async_smem();
    warp_arrive(sm.u_full[b], lane);
    // S^T = e^{G_C} S^T + (U^T diag(e^{G_C - G})) K, in a scale that both terms fit
#pragma unroll
    for (int t = 0; t < DK / 8; ++t) {
        s[t][0] *= dec[0];
        s[t][1] *= dec[0];
        s[t][2] *= dec[1];
        s[t][3] *= dec[1];
    }
    constexpr int G = DK >= 64 ? 4 : 2, NG = DK / 16 / G;  // fragments loaded at a time, and such groups in a k-tile
    auto right = [&](int step) {
#pragma unroll
        for (int t = 0; t < G; ++t)
            ldsm_t(f[step & 1][t], kb + kq_at(step / NG * 16 + trow, (step % NG * G + t) * 2 + tcol));
    };
    auto decayed = [&](int kt) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float2 w = *reinterpret_cast<const float2*>(&sm.w[b][(2 * kt + z) * 8 + q2]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* x = &u[2 * kt + z][2 * i];
                split_h(x[0] * (w.x * g[i]), x[1] * (w.y * g[i]), hi[kt & 1][2 * z + i], lo[kt & 1][2 * z + i]);
            }
        }
    };
    right(0);
    decayed(0);
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        if (kt + 1 < 4) decayed(kt + 1);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int step = kt * NG + n;
            if (step + 1 < 4 * NG) right(step + 1);
            uint32_t(&e)[4][4] = f[step & 1];
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
                mma(s[n * 2 * G + t], hi[kt & 1], e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
                mma(s[n * 2 * G + t], lo[kt & 1], e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
        }
    }
}

// ------------------------------------------------------------ outputs

// Issues the products of chunk m's outputs (one thread issues): with the rows
// of [K; Q] and [T; P] as left operands, lanes 64 - 127 hold Q S and P U.
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void issue_outputs(S& sm, int m, Waiter& wait, uint32_t tmem, int lane)
{
    const int slot = m % 3, b = m & 1;
    constexpr uint32_t id = ptx::idesc_f16(128, DVT);
    wait(sm.ready[b], m >> 1);
    wait(sm.s_full, m);
    if (m > 0) wait(sm.o_free, m - 1);
    ptx::tc_fence_after();
    if (lane == 0) {
        const uint32_t kq = ptx::smem_u32(sm.kq[slot]);
#pragma unroll 1
        for (int p = 0; p < (F32 ? 2 : 1); ++p) {
            const uint32_t st = ptx::smem_u32(sm.st[F32 ? p : 0]);
#pragma unroll 1
            for (int kt = 0; kt < DK / 16; ++kt)
                ptx::mma_f16_ss(tmem + TM_QS, ptx::desc_sw128(kq + (kt >> 2) * 16384 + (kt & 3) * 32),
                                ptx::desc_sw128(st + (kt >> 2) * DVT * 128 + (kt & 3) * 32), id, p > 0 || kt > 0);
        }
        ptx::mma_commit(&sm.s_free);
    }
    __syncwarp();
    wait(sm.u_full[b], m >> 1);
    ptx::tc_fence_after();
    if (lane == 0) {
        // T P high with U high and low, T P low with U high
        const uint32_t hi = ptx::smem_u32(sm.tp[b]), lo = hi + 16384;
#pragma unroll 1
        for (int p = 0; p < (F32 ? 3 : 1); ++p) {
            const uint32_t x = p < 2 ? hi : lo, u = ptx::smem_u32(sm.ut[F32 && p == 1 ? 1 : 0]);
#pragma unroll 1
            for (int kt = 0; kt < 4; ++kt)
                ptx::mma_f16_ss(tmem + TM_PU, ptx::desc_sw128(x + kt * 32), ptx::desc_sw128(u + kt * 32), id, p > 0 || kt > 0);
        }
        ptx::mma_commit(&sm.o_full);
    }
    __syncwarp();
}

// Rows of chunk m's outputs: o_r = scale sq (e^G q'.S + (P U)_r), a row a lane.
template <int DVT, bool F32, class S>
__device__ __forceinline__ void output_rows(S& sm, int m, void* out, long long row_stride, int n, Waiter& wait,
                                            uint32_t tmem, int half, int lane)
{
    const int b = m & 1, r = half * 32 + lane;
    wait(sm.ready[b], m >> 1);
    wait(sm.u_full[b], m >> 1);
    const float e1 = sm.e1[b][r], e2 = sm.e2[b][r];
    wait(sm.o_full, m);
    ptx::tc_fence_after();
    const uint32_t at = tmem + ((uint32_t)(64 + half * 32) << 16);
#pragma unroll 1
    for (int c0 = 0; c0 < DVT; c0 += 16) {
        float x[16], y[16];
        ptx::tmem_ld16(at + TM_QS + c0, x);
        ptx::tmem_ld16(at + TM_PU + c0, y);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 f1 = *reinterpret_cast<const float4*>(&sm.f1[b][c0 + i]);
            const float4 f2 = *reinterpret_cast<const float4*>(&sm.f2[b][c0 + i]);
            x[i] = fmaf(e1, f1.x * x[i], e2 * (f2.x * y[i]));
            x[i + 1] = fmaf(e1, f1.y * x[i + 1], e2 * (f2.y * y[i + 1]));
            x[i + 2] = fmaf(e1, f1.z * x[i + 2], e2 * (f2.z * y[i + 2]));
            x[i + 3] = fmaf(e1, f1.w * x[i + 3], e2 * (f2.w * y[i + 3]));
        }
        if (r < n) {
            if constexpr (F32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + r * row_stride + c0);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            } else {
                uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + r * row_stride + c0);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
                        v[j] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    p[i] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        __syncwarp();
    }
    ptx::tc_fence_before();
    warp_arrive(sm.o_free, lane);
}

// ------------------------------------------------------------ kernel

// The sequence of rank `rank` by length, longest first (ties: lowest index):
// long chains start first.  Up to one sequence a thread; more keep their order.
__device__ __forceinline__ int ranked_seq(const int32_t* cu, int N, int rank, int* found)
{
    if (N > (int)blockDim.x || N == 1) return rank;
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

// Sets the register count of the calling warpgroup's threads.
template <bool UP, int N> __device__ __forceinline__ void set_regs()
{
    if constexpr (UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct RowMaps {
    CUtensorMap q, k, v;
};

template <int DK, int NW, bool F32>
__global__ void __launch_bounds__(THREADS, 1) gdn_chunk_kernel(const GdnArgs a, const __grid_constant__ RowMaps maps, int dv)
{
    constexpr int DVT = NW * 16;
    extern __shared__ __align__(1024) unsigned char dyn[];
    using S = Smem<DK, DVT, F32>;
    S& sm = *reinterpret_cast<S*>(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = dv / DVT;
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % a.Hv;
    const int seq = ranked_seq(a.cu_seqlens, a.N, blockIdx.x / (parts * a.Hv), &sm.found);
    int begin, end, state_slot;
    if (!gdn_unit(a, seq, begin, end, state_slot)) return;
    const int chunks = (end - begin + C - 1) / C;
    const int col0 = part * DVT;

    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            ptx::mbar_init(&sm.loaded[i], 1);
            ptx::mbar_init(&sm.kv_free[i], NW + 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.prod_full[i], 1);
            ptx::mbar_init(&sm.prod_free[i], PREP / 32);
            ptx::mbar_init(&sm.ready[i], PREP / 32);
            ptx::mbar_init(&sm.tp_free[i], NW + 2);
            ptx::mbar_init(&sm.u_full[i], NW);
        }
        ptx::mbar_init(&sm.s_full, NW);
        ptx::mbar_init(&sm.s_free, 1);
        ptx::mbar_init(&sm.o_full, 1);
        ptx::mbar_init(&sm.o_free, 2);
        ptx::fence_mbar_init();
    }
    // P's quarter above the diagonal is read and never written
#pragma unroll 1
    for (int i = tid; i < (int)sizeof(sm.tp) / 16; i += THREADS)
        reinterpret_cast<uint4*>(sm.tp)[i] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    if (warp == 5) ptx::tmem_alloc(&sm.tmem, TM_COLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    Waiter wait{false};

    // Registers: the launch gives every thread 128; the chain's warpgroup takes
    // what the others leave (232 + 88 + 2 * 96 <= 4 * 128).
    if (warp < 4) {
        set_regs<true, 232>();
        if (warp < NW) {
            const size_t sbase = ((size_t)state_slot * a.Hv + h) * DK * dv + col0 + warp * 16 + (lane >> 2);
            float s[DK / 8][4], ig[2], ms[2] = {0.f, 0.f};
#pragma unroll
            for (int t = 0; t < DK / 8; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[t][i] = a.state[sbase + (size_t)(t * 8 + (lane & 3) * 2 + (i & 1)) * dv + (i >> 1) * 8];
                    ms[i >> 1] = fmaxf(ms[i >> 1], fabsf(s[t][i]));
                }
            {
                float g[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) pow2_scale(quad_max(ms[i]), g[i], ig[i]);
#pragma unroll
                for (int t = 0; t < DK / 8; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] *= g[i >> 1];
            }
            for (int m = 0; m < chunks; ++m) {
                wait(sm.loaded[m % 3], m / 3);
                wait(sm.ready[m & 1], m >> 1);
                chain_chunk<DK, DVT, F32>(sm, m, s, ig, wait, warp, lane);
                warp_arrive(sm.kv_free[m % 3], lane);
                if (lane == 0) ptx::mbar_arrive(&sm.tp_free[m & 1]);
            }
#pragma unroll
            for (int t = 0; t < DK / 8; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a.state[sbase + (size_t)(t * 8 + (lane & 3) * 2 + (i & 1)) * dv + (i >> 1) * 8] = s[t][i] * ig[i >> 1];
        }
    } else if (warp < PREP_WARP) {
        set_regs<false, 88>();
        if (warp == 4) {
            const int hk = h / (a.Hv / a.Hk);
            const uint64_t policy = ptx::policy_evict_normal();  // other heads and columns read the same rows
            for (int m = 0; m <= chunks; ++m) {
                if (m > 0) {
                    // the raw products of chunk m - 1
                    const int s = (m - 1) % 3, b = (m - 1) & 1;
                    wait(sm.loaded[s], (m - 1) / 3);
                    if (m >= 3) wait(sm.prod_free[b], (m - 3) >> 1);
                    ptx::tc_fence_after();
                    if (lane == 0) {
                        const uint32_t kq = ptx::smem_u32(sm.kq[s]);
#pragma unroll 1
                        for (int kt = 0; kt < DK / 16; ++kt) {
                            const uint64_t d = ptx::desc_sw128(kq + (kt >> 2) * 16384 + (kt & 3) * 32);
                            ptx::mma_f16_ss(tmem + TM_PROD + b * 128, d, d, ptx::idesc_bf16(128, 128), kt > 0);
                        }
                        ptx::mma_commit(&sm.prod_full[b]);
                    }
                    __syncwarp();
                }
                if (m < chunks) {
                    const int s = m % 3, r0 = begin + m * C;
                    if (m >= 3) wait(sm.kv_free[s], m / 3 - 1);
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(&sm.loaded[s], sizeof(sm.kq[0]) + sizeof(sm.v[0]));
#pragma unroll 1
                        for (int i = 0; i < S::HALVES; ++i) {
                            ptx::tma_load_2d(sm.kq[s] + i * 16384, &maps.k, hk * DK + i * 64, r0, &sm.loaded[s], policy);
                            ptx::tma_load_2d(sm.kq[s] + i * 16384 + 8192, &maps.q, hk * DK + i * 64, r0, &sm.loaded[s],
                                             policy);
                        }
                        ptx::tma_load_2d(sm.v[s], &maps.v, h * dv + col0, r0, &sm.loaded[s], policy);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 5) {
            for (int m = 0; m < chunks; ++m) issue_outputs<DK, DVT, F32>(sm, m, wait, tmem, lane);
        } else {
            const long long row_stride = (long long)a.Hv * dv;
            const size_t osize = F32 ? 4 : 2;
            unsigned char* out = static_cast<unsigned char*>(a.out) + ((size_t)begin * row_stride + (size_t)h * dv + col0) * osize;
            for (int m = 0; m < chunks; ++m) {
                output_rows<DVT, F32>(sm, m, out + (size_t)m * C * row_stride * osize, row_stride,
                                      min(C, end - begin - m * C), wait, tmem, warp - 6, lane);
                warp_arrive(sm.kv_free[m % 3], lane);
                if (lane == 0) ptx::mbar_arrive(&sm.tp_free[m & 1]);
            }
        }
    } else {
        set_regs<false, 96>();
        const int w = warp - PREP_WARP;
        const __nv_bfloat16* ga = static_cast<const __nv_bfloat16*>(a.a) + h;
        const __nv_bfloat16* be = static_cast<const __nv_bfloat16*>(a.b) + h;
        const float ea = expf(a.A_log[h]) * 1.44269504088896341f, dt = a.dt_bias[h];
        __nv_bfloat16 graw[2], braw[2];  // the next chunk's gates of two rows, as loaded (warp 4)
        auto gates = [&](int r0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = r0 + 2 * lane + i;
                if (w == 4 && r < end) {
                    graw[i] = ga[(size_t)r * a.Hv];
                    braw[i] = be[(size_t)r * a.Hv];
                } else graw[i] = braw[i] = __float2bfloat16(0.f);
            }
        };
        gates(begin);
        for (int m = 0; m < chunks; ++m) {
            const int r0 = begin + m * C, n = min(C, end - r0);
            float2 g = make_float2(0.f, 0.f), bt = g;
            if (w == 4) {
                if (2 * lane < n) {
                    g.x = gdn_log_alpha(ea, __bfloat162float(graw[0]), dt);
                    bt.x = sigmoidf_(__bfloat162float(braw[0]));
                }
                if (2 * lane + 1 < n) {
                    g.y = gdn_log_alpha(ea, __bfloat162float(graw[1]), dt);
                    bt.y = sigmoidf_(__bfloat162float(braw[1]));
                }
                gates(r0 + C);
            }
            prep_chunk<DK, DVT, F32>(sm, m, a, n, g, bt, wait, tmem, w, lane);
        }
    }
    if (wait.dead) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TM_COLS);
    }
}

// [T][width] bf16 rows with a row stride; boxes of 64 rows.
bool encode_rows(CUtensorMap* m, const void* base, long long width, long long stride, int T, int box)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)T};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {(cuuint32_t)box, C};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int NW, bool F32> cudaError_t launch(const GdnArgs& a, int dv, cudaStream_t st)
{
    using S = Smem<DK, NW * 16, F32>;
    // operand tiles on the swizzle's 1024-byte period, vectors on 16 bytes, barriers on 8
    static_assert(offsetof(S, v) % 1024 == 0 && offsetof(S, tp) % 1024 == 0 && offsetof(S, st) % 1024 == 0 &&
                  offsetof(S, ut) % 1024 == 0, "tiles");
    static_assert(offsetof(S, x) % 16 == 0 && offsetof(S, f1) % 16 == 0 && offsetof(S, f2) % 16 == 0 &&
                  offsetof(S, gh) % 16 == 0 && offsetof(S, gl) % 16 == 0 && offsetof(S, colk) % 16 == 0 &&
                  offsetof(S, down) % 16 == 0 && offsetof(S, loaded) % 8 == 0, "vectors");
    constexpr int smem = sizeof(Smem<DK, NW * 16, F32>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_chunk_kernel<DK, NW, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    RowMaps maps;
    if (!encode_rows(&maps.q, a.q, (long long)a.Hk * DK, a.qs, a.T, 64) ||
        !encode_rows(&maps.k, a.k, (long long)a.Hk * DK, a.ks, a.T, 64) ||
        !encode_rows(&maps.v, a.v, (long long)a.Hv * dv, a.vs, a.T, NW * 16))
        return cudaErrorInvalidValue;
    gdn_chunk_kernel<DK, NW, F32><<<a.N * a.Hv * (dv / (NW * 16)), THREADS, smem, st>>>(a, maps, dv);
    return cudaGetLastError();
}

template <int DK> cudaError_t launch_dk(const GdnArgs& a, int dv, bool bf16, cudaStream_t st)
{
    // Two chain warps a CTA where four would leave SMs without one, and where
    // the fp32 outputs' low parts take the shared memory of the other two.
    if (dv == 32 || (long long)a.N * a.Hv * (dv / 64) * 2 <= sm_count())
        return bf16 ? launch<DK, 2, false>(a, dv, st) : launch<DK, 2, true>(a, dv, st);
    if (bf16) return launch<DK, 4, false>(a, dv, st);
    return launch<DK, DK == 128 ? 2 : 4, true>(a, dv, st);
}

}  // namespace

size_t gdn_chunk_workspace_bytes(int, int, int, int, bool, int, int) { return 0; }

cudaError_t launch_gdn_chunk(const GdnArgs& a, int dk, int dv, bool out_bf16, cudaStream_t st)
{
    if (dk == 128) return launch_dk<128>(a, dv, out_bf16, st);
    if (dk == 64) return launch_dk<64>(a, dv, out_bf16, st);
    return launch_dk<32>(a, dv, out_bf16, st);
}

}  // namespace kda
