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
// columns, so these never meet.  Three roles:
//   - prep warps (4): load the chunk's rows, normalise and rescale them, form
//     P and T (state-independent), one chunk ahead of
//   - chain warps (NW): each keeps S^T for 16 columns in registers as the
//     accumulator of a 16 x dk product and walks the chunks alone: S^T K^T,
//     R^T T^T (R = beta (V - ..)) and U^T K take their left operand straight from
//     the accumulators of the product before (the two fragment layouts agree),
//     so no chain warp ever waits for another one;
//   - output warps (NW): take S^T and U^T of one chain warp each through shared
//     memory, form Q S and P U and store the outputs beside the chain.
//
// Precision: the state keeps fp32 accuracy.  One decay per head leaves k and q
// unscaled inside every product, so the rows' bf16 values are operands without
// loss: prep rescales each row by a power of two to a norm in [1, 2) and stores
// it as fp16 (exact down to 2^-17).  Every other operand that
// reaches the state is two fp16 values, high and low, about 22 bits: S and
// U and V - .. are scaled by a power of two per column so that the low part stays
// in fp16's range.  P and the outputs' reading of S keep the high part only
// where the outputs are bf16 (11 bits against their 8).
#include <cuda_fp16.h>

#include "kda_gdn.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int C = 64;
constexpr int PREP = 128;  // prep threads
constexpr int XS = 72;     // row stride of the fp32 scratch: fragment reads hit distinct banks

// ------------------------------------------------------------ fragments

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same on bf16 values
__device__ __forceinline__ void mma_bf(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
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

// Byte offset of 16-byte piece `c` of row `r` in a tile of W 16-bit values a
// row: pieces permuted within the row so that eight rows' same piece lie in
// distinct banks.
template <int W> __device__ __forceinline__ uint32_t at(int r, int c)
{
    if constexpr (W >= 64) return (uint32_t)(r * (W * 2) + (((c & ~7) | ((c ^ r) & 7)) << 4));
    else return (uint32_t)(r * (W * 2) + ((c ^ ((r >> 1) & 3)) << 4));
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

// ------------------------------------------------------------ shared memory

template <int DK, int DVT, bool F32> struct Smem {
    static constexpr int NW = DVT / 16, PARTS = F32 ? 2 : 1;
    unsigned char k[3][C * DK * 2];        // bf16 rows, then fp16
    unsigned char q[3][C * DK * 2];
    unsigned char v[3][C * DVT * 2];       // bf16; an output warp's columns take its outputs afterwards
    unsigned char t[2][2][C * C * 2];      // T, high and low
    unsigned char p[2][PARTS][C * C * 2];
    uint4 hs[NW][PARTS][DK / 16][32];      // S^T as left-operand fragments, from a chain warp to its output warp
    uint4 hu[NW][PARTS][4][32];            // U^T likewise
    float4 hf[NW][8];                      // and their scales
    float x[C * XS];                       // A, then T, in fp32
    // per chunk row: beta; beta sk e^G; sk; e^{G_C - G}; e^G; scale sq
    float beta[2][C], ek[2][C], sk[2][C], w[2][C], eg[2][C], oq[2][C];
    float last[2];                         // e^{G_C}
    float g[C], gh[C], gl[C], bk[C], nk[C], nq[C];
    uint64_t ready[2], done[2];            // a chunk's operands; their last use
    uint64_t s_full[NW], s_free[NW], u_full[NW], u_free[NW];
};

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, %0;" ::"n"(PREP) : "memory"); }

// ------------------------------------------------------------ prep

// Starts the copies of a tile of W-wide rows r0 .. r0 + n - 1 (rows past n:
// zeros).  A thread keeps its 16-byte piece and steps down the rows.
template <int W>
__device__ __forceinline__ void load_tile(unsigned char* tile, const __nv_bfloat16* src, long long stride, int n, int t)
{
    constexpr int P = W / 8, RS = PREP / P;  // pieces of a row; rows between a thread's pieces
    static_assert(C % RS == 0 && RS % 8 == 0, "the swizzle repeats every eight rows");
    const int r = t / P, c = t % P;
    const __nv_bfloat16* s = src + r * stride + c * 8;
    unsigned char* d = tile + at<W>(r, c);
#pragma unroll
    for (int i = 0; i < C / RS; ++i) {
        const bool in = r + i * RS < n;
        ptx::cp_async16(d + i * RS * W * 2, in ? s + (long long)i * RS * stride : src, in ? 16 : 0);
    }
}

// (h, l) += (oh, ol) in double-word fp32
__device__ __forceinline__ void dw_add(float& h, float& l, float oh, float ol)
{
    const float s = __fadd_rn(h, oh), bb = __fsub_rn(s, h);
    const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(s, bb)), __fsub_rn(oh, bb));
    const float r = __fadd_rn(__fadd_rn(l, ol), e);
    h = __fadd_rn(s, r);
    l = __fsub_rn(r, __fsub_rn(h, s));
}

// One warp: running sums of the chunk's log decays, two rows a lane (double
// word: differences of large sums keep their small part).
template <class S> __device__ __forceinline__ void scan_rows(S& sm, int b, int lane)
{
    const float2 g = *reinterpret_cast<const float2*>(&sm.g[2 * lane]);
    float h = g.x, l = 0.f;
    dw_add(h, l, g.y, 0.f);
#pragma unroll
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
    *reinterpret_cast<float2*>(&sm.eg[b][2 * lane]) = make_float2(exp_sfu(ph + pl), exp_sfu(h + l));
    *reinterpret_cast<float2*>(&sm.w[b][2 * lane]) =
        make_float2(exp_sfu((th - ph) + (tl - pl)), exp_sfu((th - h) + (tl - l)));
    if (lane == 0) sm.last[b] = exp_sfu(th + tl);
}

// One row of a tile: bf16 -> fp16 times a power of two, in place.
template <int DK> __device__ __forceinline__ void convert_row(unsigned char* tile, int r, float down)
{
    const __nv_bfloat162 d = __float2bfloat162_rn(down);
#pragma unroll
    for (int c = 0; c < DK / 8; ++c) {
        uint4* p = reinterpret_cast<uint4*>(tile + at<DK>(r, c));
        const uint4 x = *p;
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), d);
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
            w[i] = pack_h(bf_lo(u), bf_hi(u));
        }
        *p = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The panel of 16 columns n0 of  T21 = -T22 (A21 T11)  for the SIZE-blocks at
// (i0, j0) of the scratch, its 16-row part `mt`; all operands split in two.
template <int SIZE, class S> __device__ __forceinline__ void merge_panel(S& sm, int b, int i0, int j0, int n0, int mt, int lane)
{
    const int gq = lane >> 2, q2 = (lane & 3) * 2;
    const float* X = sm.x;
    float pt[SIZE / 8][4];  // (A21 T11)^T, rows n
#pragma unroll
    for (int t = 0; t < SIZE / 8; ++t) pt[t][0] = pt[t][1] = pt[t][2] = pt[t][3] = 0.f;
#pragma unroll
    for (int kt = 0; kt < SIZE / 16; ++kt) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = j0 + n0 + gq + (i & 1) * 8, j = j0 + kt * 16 + q2 + (i >> 1) * 8;
            split_h(X[j * XS + n], X[(j + 1) * XS + n], ah[i], al[i]);
        }
#pragma unroll
        for (int t = 0; t < SIZE / 8; ++t) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f = *reinterpret_cast<const float2*>(&X[(i0 + t * 8 + gq) * XS + j0 + kt * 16 + q2 + i * 8]);
                split_h(f.x, f.y, bh[i], bl[i]);
            }
            mma(pt[t], ah, bh[0], bh[1]);
            mma(pt[t], ah, bl[0], bl[1]);
            mma(pt[t], al, bh[0], bh[1]);
        }
    }
    float o[2][4] = {};
#pragma unroll
    for (int kt = 0; kt < SIZE / 16; ++kt) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2*>(
                &X[(i0 + mt * 16 + gq + (i & 1) * 8) * XS + i0 + kt * 16 + q2 + (i >> 1) * 8]);
            split_h(f.x, f.y, ah[i], al[i]);
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            uint32_t bh[2], bl[2];
            split_h(pt[2 * kt][2 * nt], pt[2 * kt][2 * nt + 1], bh[0], bl[0]);
            split_h(pt[2 * kt + 1][2 * nt], pt[2 * kt + 1][2 * nt + 1], bh[1], bl[1]);
            mma(o[nt], ah, bh[0], bh[1]);
            mma(o[nt], ah, bl[0], bl[1]);
            mma(o[nt], al, bh[0], bh[1]);
        }
    }
    // the merged blocks: into the operand tiles, and for the next size into the scratch
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i0 + mt * 16 + gq + i * 8, s = j0 + n0 + nt * 8 + q2;
            const float x = -o[nt][2 * i], y = -o[nt][2 * i + 1];
            if (SIZE == 16) *reinterpret_cast<float2*>(&sm.x[r * XS + s]) = make_float2(x, y);
            uint32_t hi, lo;
            split_h(x, y, hi, lo);
            *reinterpret_cast<uint32_t*>(sm.t[b][0] + at<C>(r, s >> 3) + (s & 7) * 2) = hi;
            *reinterpret_cast<uint32_t*>(sm.t[b][1] + at<C>(r, s >> 3) + (s & 7) * 2) = lo;
        }
}

// The 16 x 16 blocks on and below the diagonal, by warp: two or three each.
__device__ __forceinline__ void block_of(int warp, int j, int& bi, int& bj)
{
    // (3,0) (3,1) (0,0) | (3,2) (3,3) (1,1) | (2,0) (2,1) | (2,2) (1,0)
    const int i = warp * 3 + j;
    bi = (int)((0b00'01'10'00'10'10'01'11'11'00'11'11u >> (2 * i)) & 3);
    bj = (int)((0b00'00'10'00'01'00'01'11'10'00'01'00u >> (2 * i)) & 3);
}

// The chunk's P and T into buffer b from the rows in slot `slot`; g, beta: the
// log decay and beta of row t & 63 (zero for a padded row).
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void prep_chunk(S& sm, int slot, int b, const GdnArgs& a, bool real, int t)
{
    const int warp = t >> 5, lane = t & 31, gq = lane >> 2, q2 = (lane & 3) * 2;
    if (warp == 3) scan_rows(sm, b, lane);
    // K K^T and Q K^T of the raw rows: bf16 values, exact products
    const uint32_t kb = ptx::smem_u32(sm.k[slot]), qb = ptx::smem_u32(sm.q[slot]);
    const int arow = lane & 15, acol = lane >> 4, brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
    float kk[3][2][4], qk[3][2][4];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if (j == 2 && warp >= 2) break;
        int bi, bj;
        block_of(warp, j, bi, bj);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) kk[j][n][i] = qk[j][n][i] = 0.f;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t ka[4], qa[4], bb[4];
            const uint32_t ao = at<DK>(bi * 16 + arow, kt * 2 + acol);
            ldsm(ka, kb + ao);
            ldsm(qa, qb + ao);
            ldsm(bb, kb + at<DK>(bj * 16 + brow, kt * 2 + bcol));
            mma_bf(kk[j][0], ka, bb[0], bb[1]);
            mma_bf(kk[j][1], ka, bb[2], bb[3]);
            mma_bf(qk[j][0], qa, bb[0], bb[1]);
            mma_bf(qk[j][1], qa, bb[2], bb[3]);
        }
        if (bi == bj) {  // squared norms of k's rows
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (q2 == gq) sm.nk[bi * 16 + i * 8 + gq] = kk[j][i][2 * i];
                if (q2 + 1 == gq) sm.nk[bi * 16 + i * 8 + gq] = kk[j][i][2 * i + 1];
            }
        }
    }
    {
        // and of q's
        float qq[2][4] = {};
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t qa[4], bb[4];
            ldsm(qa, qb + at<DK>(warp * 16 + arow, kt * 2 + acol));
            ldsm(bb, qb + at<DK>(warp * 16 + brow, kt * 2 + bcol));
            mma_bf(qq[0], qa, bb[0], bb[1]);
            mma_bf(qq[1], qa, bb[2], bb[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (q2 == gq) sm.nq[warp * 16 + i * 8 + gq] = qq[i][2 * i];
            if (q2 + 1 == gq) sm.nq[warp * 16 + i * 8 + gq] = qq[i][2 * i + 1];
        }
    }
    prep_sync();
    {
        const int r = t & (C - 1);
        const float ss = t < C ? sm.nk[r] : sm.nq[r];
        float down, up;
        pow2_scale_sqrt(ss, down, up);
        // the factor that makes the stored row the (normalised) row; none for a padded one
        const float norm = a.l2 ? rsqrtf(ss + a.l2_eps) : 1.f;
        if (t < C) {
            const float f = real ? norm * up : 0.f, e = sm.eg[b][r];
            sm.sk[b][r] = f;
            sm.ek[b][r] = sm.beta[b][r] * f * e;
            sm.nk[r] = real ? norm : 0.f;               // raw rows enter A and P
            sm.bk[r] = real ? sm.beta[b][r] * norm : 0.f;
        } else sm.oq[b][r] = real ? a.scale * norm * up : 0.f;
        if (t >= C) sm.nq[r] = down;
        convert_row<DK>(t < C ? sm.k[slot] : sm.q[slot], r, down);
        // P = e^{G_r - G_s} q'_r.k'_s on the stored rows' scale: k's part
        if (t < C) sm.g[r] = down;
    }
    prep_sync();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if (j == 2 && warp >= 2) break;
        int bi, bj;
        block_of(warp, j, bi, bj);
        float2 ch[2], cl[2], cn[2], cd[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int s = bj * 16 + n * 8 + q2;
            ch[n] = *reinterpret_cast<const float2*>(&sm.gh[s]);
            cl[n] = *reinterpret_cast<const float2*>(&sm.gl[s]);
            cn[n] = *reinterpret_cast<const float2*>(&sm.nk[s]);
            cd[n] = *reinterpret_cast<const float2*>(&sm.g[s]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = bi * 16 + gq + i * 8;
            const float rh = sm.gh[r], rl = sm.gl[r], br = sm.bk[r], qd = sm.nq[r];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int s = bj * 16 + n * 8 + q2;
                const float d0 = exp_sfu((rh - ch[n].x) + (rl - cl[n].x)), d1 = exp_sfu((rh - ch[n].y) + (rl - cl[n].y));
                const float a0 = s < r ? (br * cn[n].x) * d0 * kk[j][n][2 * i] : 0.f;
                const float a1 = s + 1 < r ? (br * cn[n].y) * d1 * kk[j][n][2 * i + 1] : 0.f;
                const float p0 = s <= r ? (qd * cd[n].x) * d0 * qk[j][n][2 * i] : 0.f;
                const float p1 = s + 1 <= r ? (qd * cd[n].y) * d1 * qk[j][n][2 * i + 1] : 0.f;
                *reinterpret_cast<float2*>(&sm.x[r * XS + s]) = make_float2(a0, a1);
                const uint32_t o = at<C>(r, s >> 3) + (s & 7) * 2;
                if constexpr (F32) {
                    uint32_t hi, lo;
                    split_h(p0, p1, hi, lo);
                    *reinterpret_cast<uint32_t*>(sm.p[b][0] + o) = hi;
                    *reinterpret_cast<uint32_t*>(sm.p[b][1] + o) = lo;
                } else *reinterpret_cast<uint32_t*>(sm.p[b][0] + o) = pack_h(p0, p1);
            }
        }
    }
    prep_sync();
    {
        // the diagonal block of each warp: forward substitution, a column a lane
        const int d0 = warp * 16, c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == c ? 1.f : 0.f, acc2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sm.x[(d0 + i) * XS + d0 + m]);
                acc = fmaf(-f.x, x[m], acc);
                if (m + 1 < i) acc2 = fmaf(-f.y, x[m + 1], acc2);
                if (m + 2 < i) acc = fmaf(-f.z, x[m + 2], acc);
                if (m + 3 < i) acc2 = fmaf(-f.w, x[m + 3], acc2);
            }
            x[i] = acc + acc2;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sm.x[(d0 + i) * XS + d0 + c] = x[i];
                const __half hi = __float2half_rn(x[i]);
                const uint32_t o = at<C>(d0 + i, (d0 + c) >> 3) + (c & 7) * 2;
                *reinterpret_cast<__half*>(sm.t[b][0] + o) = hi;
                *reinterpret_cast<__half*>(sm.t[b][1] + o) = __float2half_rn(x[i] - __half2float(hi));
            }
        }
    }
    prep_sync();
    if (warp < 2) merge_panel<16>(sm, b, 16 + warp * 32, warp * 32, 0, 0, lane);
    prep_sync();
    merge_panel<32>(sm, b, 32, 0, (warp & 1) * 16, warp >> 1, lane);
}

// ------------------------------------------------------------ chain

// A bounded wait that gives up once: later ones are skipped, the status word says so.
struct Waiter {
    int32_t* dev_status;
    bool dead;
    __device__ __forceinline__ void operator()(uint64_t& bar, int phase)
    {
        if (!dead && !ptx::mbar_wait(&bar, phase & 1)) {
            dead = true;
            flag_status(dev_status, KDA_DEV_TIMEOUT);
        }
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

// Chunk m of a chain warp: 16 columns of dv.  s holds S^T times g[0] (column
// lane / 4) and g[1] (eight further), ig their inverses.
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void chain_chunk(S& sm, int m, float (&s)[DK / 8][4], float (&ig)[2], Waiter& wait, int warp,
                                            int lane)
{
    const int slot = m % 3, b = m & 1, q2 = (lane & 3) * 2;
    const uint32_t kb = ptx::smem_u32(sm.k[slot]), vb = ptx::smem_u32(sm.v[slot]);
    const uint32_t tb[2] = {ptx::smem_u32(sm.t[b][0]), ptx::smem_u32(sm.t[b][1])};
    const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;  // K-contiguous operand
    const int trow = lane & 15, tcol = lane >> 4;                                 // transposed operand
    if (m > 0) wait(sm.s_free[warp], m - 1);

    // S^T K^T, each k-tile's fragments loaded a tile ahead
    float r[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[t][i] = 0.f;
    __half2 m0 = __float2half2_rn(0.f), m1 = m0;
    uint32_t f[2][4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) ldsm(f[0][t], kb + at<DK>(t * 16 + brow, bcol));
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        if (kt + 1 < DK / 16)
#pragma unroll
            for (int t = 0; t < 4; ++t) ldsm(f[(kt + 1) & 1][t], kb + at<DK>(t * 16 + brow, (kt + 1) * 2 + bcol));
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = &s[2 * kt + (i >> 1)][2 * (i & 1)];
            split_h(x[0], x[1], hi[i], lo[i]);
            const __half2 h = __habs2(*reinterpret_cast<const __half2*>(&hi[i]));
            if (i & 1) m1 = __hmax2(m1, h);
            else m0 = __hmax2(m0, h);
        }
        sm.hs[warp][0][kt][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (F32) sm.hs[warp][F32 ? 1 : 0][kt][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        uint32_t(&e)[4][4] = f[kt & 1];
#pragma unroll
        for (int t = 0; t < 8; ++t) mma(r[t], hi, e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 8; ++t) mma(r[t], lo, e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
    }
    warp_arrive(sm.s_full[warp], lane);
    // beta (V - e^G k.S), and each column's largest value
    float mr[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
        uint32_t v[4];  // V^T: rows t*8.. of columns gq, gq+8; then the next eight rows
        ldsm_t(v, vb + at<DVT>(t * 8 + brow, warp * 2 + bcol));
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
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t hi[4], lo[4], th[4][4], tl[4][4];
#pragma unroll
        for (int t = kt; t < 4; ++t) {
            ldsm(th[t], tb[0] + at<C>(t * 16 + brow, kt * 2 + bcol));
            ldsm(tl[t], tb[1] + at<C>(t * 16 + brow, kt * 2 + bcol));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = &r[2 * kt + (i >> 1)][2 * (i & 1)];
            split_h(x[0] * rd[i & 1], x[1] * rd[i & 1], hi[i], lo[i]);
        }
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], hi, th[t >> 1][2 * (t & 1)], th[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], lo, th[t >> 1][2 * (t & 1)], th[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(u[t], hi, tl[t >> 1][2 * (t & 1)], tl[t >> 1][2 * (t & 1) + 1]);
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
        float old[2] = {ig[0], ig[1]}, up;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // 2^-20: keeps the outputs' S term in range beside a tiny U
            pow2_scale(quad_max(fmaxf(mu[i], ms[i] * 0x1p-20f)), ud[i], up);
            pow2_scale(quad_max(fmaxf(mw[i], ms[i] * last)), g[i], ig[i]);
            dec[i] = last * (g[i] * old[i]);
        }
        if (m > 0) wait(sm.u_free[warp], m - 1);
        if ((lane & 3) == 0) sm.hf[warp][lane >> 2] = make_float4(ud[0], ud[1], old[0], old[1]);
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = &u[2 * kt + (i >> 1)][2 * (i & 1)];
            if (F32) split_h(x[0] * ud[i & 1], x[1] * ud[i & 1], hi[i], lo[i]);
            else hi[i] = pack_h(x[0] * ud[i & 1], x[1] * ud[i & 1]);
        }
        sm.hu[warp][0][kt][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (F32) sm.hu[warp][F32 ? 1 : 0][kt][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    warp_arrive(sm.u_full[warp], lane);
    // S^T = e^{G_C} S^T + (U^T diag(e^{G_C - G})) K, in a scale that both terms fit
#pragma unroll
    for (int t = 0; t < DK / 8; ++t) {
        s[t][0] *= dec[0];
        s[t][1] *= dec[0];
        s[t][2] *= dec[1];
        s[t][3] *= dec[1];
    }
    constexpr int G = DK >= 64 ? 4 : 2, NG = DK / 16 / G;  // fragments loaded at a time, and such groups in a k-tile
#pragma unroll
    for (int t = 0; t < G; ++t) ldsm_t(f[0][t], kb + at<DK>(trow, t * 2 + tcol));
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float2 w = *reinterpret_cast<const float2*>(&sm.w[b][(2 * kt + z) * 8 + q2]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* x = &u[2 * kt + z][2 * i];
                split_h(x[0] * (w.x * g[i]), x[1] * (w.y * g[i]), hi[2 * z + i], lo[2 * z + i]);
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int step = kt * NG + n;
            if (step + 1 < 4 * NG)
#pragma unroll
                for (int t = 0; t < G; ++t)
                    ldsm_t(f[(step + 1) & 1][t],
                           kb + at<DK>((step + 1) / NG * 16 + trow, ((step + 1) % NG * G + t) * 2 + tcol));
            uint32_t(&e)[4][4] = f[step & 1];
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) mma(s[n * 2 * G + t], hi, e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) mma(s[n * 2 * G + t], lo, e[t >> 1][2 * (t & 1)], e[t >> 1][2 * (t & 1) + 1]);
        }
    }
}

// Chunk m of an output warp, from its chain warp's fragments:
// O^T = scale sq (e^G S^T Q^T + U^T P^T).
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void output_chunk(S& sm, int m, void* out, long long row_stride, int n, Waiter& wait, int warp,
                                             int lane)
{
    const int slot = m % 3, b = m & 1, q2 = (lane & 3) * 2;
    const uint32_t qb = ptx::smem_u32(sm.q[slot]), vb = ptx::smem_u32(sm.v[slot]);
    const uint32_t pb[2] = {ptx::smem_u32(sm.p[b][0]), ptx::smem_u32(sm.p[b][F32 ? 1 : 0])};
    const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
    float o[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    wait(sm.s_full[warp], m);
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        const uint4 h4 = sm.hs[warp][0][kt][lane];
        const uint32_t hi[4] = {h4.x, h4.y, h4.z, h4.w};
        uint4 l4 = h4;
        if (F32) l4 = sm.hs[warp][F32 ? 1 : 0][kt][lane];
        const uint32_t lo[4] = {l4.x, l4.y, l4.z, l4.w};
        uint32_t f[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) ldsm(f[t], qb + at<DK>(t * 16 + brow, kt * 2 + bcol));
#pragma unroll
        for (int t = 0; t < 8; ++t) mma(o[t], hi, f[t >> 1][2 * (t & 1)], f[t >> 1][2 * (t & 1) + 1]);
        if (F32)
#pragma unroll
            for (int t = 0; t < 8; ++t) mma(o[t], lo, f[t >> 1][2 * (t & 1)], f[t >> 1][2 * (t & 1) + 1]);
    }
    warp_arrive(sm.s_free[warp], lane);
    wait(sm.u_full[warp], m);
    const float4 sc = sm.hf[warp][lane >> 2];
    const float ud[2] = {sc.x, sc.y}, fs[2] = {sc.x * sc.z, sc.y * sc.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float2 eg = *reinterpret_cast<const float2*>(&sm.eg[b][t * 8 + q2]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[t][2 * i] *= eg.x * fs[i];
            o[t][2 * i + 1] *= eg.y * fs[i];
        }
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        const uint4 h4 = sm.hu[warp][0][kt][lane];
        const uint32_t hi[4] = {h4.x, h4.y, h4.z, h4.w};
        uint4 l4 = h4;
        if (F32) l4 = sm.hu[warp][F32 ? 1 : 0][kt][lane];
        const uint32_t lo[4] = {l4.x, l4.y, l4.z, l4.w};
        uint32_t f[4][4];
#pragma unroll
        for (int t = kt; t < 4; ++t) ldsm(f[t], pb[0] + at<C>(t * 16 + brow, kt * 2 + bcol));
#pragma unroll
        for (int t = 2 * kt; t < 8; ++t) mma(o[t], hi, f[t >> 1][2 * (t & 1)], f[t >> 1][2 * (t & 1) + 1]);
        if (F32) {
#pragma unroll
            for (int t = 2 * kt; t < 8; ++t) mma(o[t], lo, f[t >> 1][2 * (t & 1)], f[t >> 1][2 * (t & 1) + 1]);
#pragma unroll
            for (int t = kt; t < 4; ++t) ldsm(f[t], pb[1] + at<C>(t * 16 + brow, kt * 2 + bcol));
#pragma unroll
            for (int t = 2 * kt; t < 8; ++t) mma(o[t], hi, f[t >> 1][2 * (t & 1)], f[t >> 1][2 * (t & 1) + 1]);
        }
    }
    warp_arrive(sm.u_free[warp], lane);
    float uu[2];  // 1 / ud: a power of two
#pragma unroll
    for (int i = 0; i < 2; ++i) uu[i] = __uint_as_float((254u << 23) - __float_as_uint(ud[i]));
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float2 oq = *reinterpret_cast<const float2*>(&sm.oq[b][t * 8 + q2]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[t][2 * i] *= oq.x * uu[i];
            o[t][2 * i + 1] *= oq.y * uu[i];
        }
    }
    if constexpr (F32) {
        float* op = static_cast<float*>(out) + warp * 16 + (lane >> 2);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int z = 0; z < 2; ++z)
                if (t * 8 + q2 + z < n) {
                    float* p = op + (t * 8 + q2 + z) * row_stride;
                    p[0] = o[t][z];
                    p[8] = o[t][2 + z];
                }
    } else {
        // through the warp's own columns of the V tile: 32 bytes a row to global memory
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[t + (i >> 1)][2 * (i & 1)], o[t + (i >> 1)][2 * (i & 1) + 1]);
                f[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            stsm_t(vb + at<DVT>(t * 8 + brow, warp * 2 + bcol), f[0], f[1], f[2], f[3]);
        }
        __syncwarp();
        __nv_bfloat16* op = static_cast<__nv_bfloat16*>(out) + warp * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = lane + 32 * j, rr = i >> 1, c = i & 1;
            if (rr < n)
                *reinterpret_cast<uint4*>(op + rr * row_stride + c * 8) =
                    *reinterpret_cast<const uint4*>(sm.v[slot] + at<DVT>(rr, warp * 2 + c));
        }
    }
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

template <int DK, int NW, bool F32>
__global__ void __launch_bounds__(NW * 64 + PREP, 1) gdn_chunk_kernel(const GdnArgs a, int dv)
{
    constexpr int DVT = NW * 16, THREADS = NW * 64 + PREP;
    extern __shared__ __align__(1024) unsigned char dyn[];
    using S = Smem<DK, DVT, F32>;
    S& sm = *reinterpret_cast<S*>(dyn);
    __shared__ int found;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = dv / DVT;
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % a.Hv;
    const int seq = ranked_seq(a.cu_seqlens, a.N, blockIdx.x / (parts * a.Hv), &found);
    int begin, end, slot;
    if (!gdn_unit(a, seq, begin, end, slot)) return;
    const int chunks = (end - begin + C - 1) / C;
    const int col0 = part * DVT;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.ready[i], PREP);
            ptx::mbar_init(&sm.done[i], 2 * NW);
        }
        for (int i = 0; i < NW; ++i) {
            ptx::mbar_init(&sm.s_full[i], 1);
            ptx::mbar_init(&sm.s_free[i], 1);
            ptx::mbar_init(&sm.u_full[i], 1);
            ptx::mbar_init(&sm.u_free[i], 1);
        }
        ptx::fence_mbar_init();
    }
    for (int i = tid; i < C * XS; i += THREADS) sm.x[i] = 0.f;  // blocks above the diagonal stay zero
    __syncthreads();
    Waiter wait{a.dev_status, false};

    if (warp >= 2 * NW) {
        const int t = tid - NW * 64, hk = h / (a.Hv / a.Hk);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + hk * DK;
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + hk * DK;
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + h * dv + col0;
        const __nv_bfloat16* ga = static_cast<const __nv_bfloat16*>(a.a) + h;
        const __nv_bfloat16* be = static_cast<const __nv_bfloat16*>(a.b) + h;
        const float a_log = a.A_log[h], dt = a.dt_bias[h];
        float graw = 0.f, braw = 0.f;
        auto load = [&](int m) {
            const int r0 = begin + m * C, n = min(C, end - r0), s = m % 3, r = r0 + (t & (C - 1));
            load_tile<DK>(sm.k[s], k + r0 * a.ks, a.ks, n, t);
            load_tile<DK>(sm.q[s], q + r0 * a.qs, a.qs, n, t);
            load_tile<DVT>(sm.v[s], v + r0 * a.vs, a.vs, n, t);
            ptx::cp_async_commit();
            if (t < C && r < end) {
                graw = ldv(ga + (size_t)r * a.Hv);
                braw = ldv(be + (size_t)r * a.Hv);
            }
        };
        load(0);
        for (int m = 0; m < chunks; ++m) {
            const int b = m & 1;
            const bool real = begin + m * C + (t & (C - 1)) < end;
            const float g0 = graw, b0 = braw;
            if (m >= 2) wait(sm.done[b], (m - 2) >> 1);
            if (t < C) {
                sm.g[t] = real ? gdn_log_alpha(a_log, g0, dt) : 0.f;
                sm.beta[b][t] = real ? sigmoidf_(b0) : 0.f;
            }
            if (m + 1 < chunks) {
                load(m + 1);
                ptx::cp_async_wait_prev();
            } else ptx::cp_async_wait_all();
            prep_sync();
            prep_chunk<DK, DVT, F32>(sm, m % 3, b, a, real, t);
            ptx::mbar_arrive(&sm.ready[b]);
            prep_sync();  // the scratch and the decays are free again
        }
        return;
    }

    if (warp >= NW) {
        const int w = warp - NW;
        const long long row_stride = (long long)a.Hv * dv;
        const size_t osize = F32 ? 4 : 2;
        unsigned char* out = static_cast<unsigned char*>(a.out) + ((size_t)begin * row_stride + (size_t)h * dv + col0) * osize;
        for (int m = 0; m < chunks; ++m) {
            wait(sm.ready[m & 1], m >> 1);
            output_chunk<DK, DVT, F32>(sm, m, out + (size_t)m * C * row_stride * osize, row_stride,
                                       min(C, end - begin - m * C), wait, w, lane);
            warp_arrive(sm.done[m & 1], lane);
        }
        return;
    }

    const size_t sbase = ((size_t)slot * a.Hv + h) * DK * dv + col0 + warp * 16 + (lane >> 2);
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
        wait(sm.ready[m & 1], m >> 1);
        chain_chunk<DK, DVT, F32>(sm, m, s, ig, wait, warp, lane);
        warp_arrive(sm.done[m & 1], lane);
    }
#pragma unroll
    for (int t = 0; t < DK / 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a.state[sbase + (size_t)(t * 8 + (lane & 3) * 2 + (i & 1)) * dv + (i >> 1) * 8] = s[t][i] * ig[i >> 1];
}

template <int DK, int NW, bool F32> cudaError_t launch(const GdnArgs& a, int dv, cudaStream_t st)
{
    constexpr int smem = sizeof(Smem<DK, NW * 16, F32>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_chunk_kernel<DK, NW, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    gdn_chunk_kernel<DK, NW, F32><<<a.N * a.Hv * (dv / (NW * 16)), NW * 64 + PREP, smem, st>>>(a, dv);
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
