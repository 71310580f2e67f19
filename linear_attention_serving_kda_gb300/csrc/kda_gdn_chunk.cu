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
//   - prep warps (8): load the chunk's rows, normalise and rescale them, form
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
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kda_gdn.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int C = 64;
constexpr int PREP = 256;  // prep threads
constexpr int XS = 20;     // row stride of the fp32 diagonal blocks

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

// Byte offset of 16-byte piece `c` of row `r` in a tile of 64 rows of W 16-bit
// values, as a tensor copy with 128-byte (W >= 64: 64 values a row, one such
// tile after the other) or 64-byte (W = 32) swizzle leaves it: eight rows' same
// piece lie in distinct banks.
template <int W> __device__ __forceinline__ uint32_t at(int r, int c)
{
    if constexpr (W >= 64) return (uint32_t)((c >> 3) * (C * 128) + r * 128 + (((c ^ r) & 7) << 4));
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
    float x[C * XS];                       // A's diagonal blocks, 16 x 16 each
    // per chunk row: beta; beta sk e^G; sk; e^{G_C - G}; e^G; scale sq
    float beta[2][C], ek[2][C], sk[2][C], w[2][C], eg[2][C], oq[2][C];
    float last[2];                         // e^{G_C}
    float g[C], gh[C], gl[C], bk[C], nk[C], nq[C];
    uint64_t loaded[3], ready[2], done[2]; // a chunk's rows; its operands; their last use
    int found;
    uint64_t s_full[NW], s_free[NW], u_full[NW], u_free[NW];
};

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, %0;" ::"n"(PREP) : "memory"); }

// ------------------------------------------------------------ prep

// Starts the copy of 64 rows from row r0, W values from column x, of a row
// tensor (rows past the tensor: zeros).
template <int W>
__device__ __forceinline__ void load_tile(unsigned char* tile, const CUtensorMap* map, int x, int r0, uint64_t* bar,
                                          uint64_t policy)
{
    constexpr int B = W >= 64 ? 64 : W;  // values a box is wide
#pragma unroll
    for (int i = 0; i < W / B; ++i) ptx::tma_load_2d(tile + i * C * B * 2, map, x + i * B, r0, bar, policy);
}

template <int W> __device__ __forceinline__ void zero_row(unsigned char* tile, int r)
{
#pragma unroll 1
    for (int c = 0; c < W / 8; ++c) *reinterpret_cast<uint4*>(tile + at<W>(r, c)) = make_uint4(0, 0, 0, 0);
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
    *reinterpret_cast<float2*>(&sm.eg[b][2 * lane]) = make_float2(exp_sfu(ph + pl), exp_sfu(h + l));
    *reinterpret_cast<float2*>(&sm.w[b][2 * lane]) =
        make_float2(exp_sfu((th - ph) + (tl - pl)), exp_sfu((th - h) + (tl - l)));
    if (lane == 0) sm.last[b] = exp_sfu(th + tl);
}

// Half a row of a tile: bf16 -> fp16 times a power of two, in place.
template <int DK> __device__ __forceinline__ void convert_row(unsigned char* tile, int r, int half, float down)
{
    const __nv_bfloat162 d = __float2bfloat162_rn(down);
    constexpr int P = DK / 16 < 4 ? DK / 16 : 4;  // pieces in flight
#pragma unroll
    for (int c0 = 0; c0 < DK / 16; c0 += P) {
        uint4 x[P];
#pragma unroll
        for (int c = 0; c < P; ++c) x[c] = *reinterpret_cast<const uint4*>(tile + at<DK>(r, half * (DK / 16) + c0 + c));
#pragma unroll
        for (int c = 0; c < P; ++c) {
            uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), d);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
                w[i] = pack_h(bf_lo(u), bf_hi(u));
            }
            x[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(tile + at<DK>(r, half * (DK / 16) + c0 + c)) = x[c];
    }
}

// x, y as fp16 high and low pairs at (r, s), (r, s + 1) of two operand tiles
__device__ __forceinline__ void put_pair(unsigned char* hi_tile, unsigned char* lo_tile, int r, int s, float x, float y)
{
    uint32_t hi, lo;
    split_h(x, y, hi, lo);
    const uint32_t o = at<C>(r, s >> 3) + (s & 7) * 2;
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
        const uint32_t th = ptx::smem_u32(sm.t[b][0]), tl = ptx::smem_u32(sm.t[b][1]);
        const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
#pragma unroll
        for (int t = 0; t < SIZE / 8; ++t) pt[t][0] = pt[t][1] = pt[t][2] = pt[t][3] = 0.f;
#pragma unroll
        for (int kt = 0; kt < SIZE / 16; ++kt) {
            uint32_t ah[4], al[4], bh[SIZE / 16][4], bl[SIZE / 16][4];
            const uint32_t ao = at<C>(j0 + kt * 16 + brow, ((j0 + n0) >> 3) + bcol);
            ldsm_t(ah, th + ao);
            ldsm_t(al, tl + ao);
#pragma unroll
            for (int t = 0; t < SIZE / 16; ++t) {
                const uint32_t bo = at<C>(i0 + t * 16 + brow, ((j0 + kt * 16) >> 3) + bcol);
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
        const uint32_t th = ptx::smem_u32(sm.t[b][0]), tl = ptx::smem_u32(sm.t[b][1]);
#pragma unroll
        for (int n = 0; n < 2; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
        for (int kt = 0; kt < SIZE / 16; ++kt) {
            uint32_t ah[4], al[4], bh[2][2], bl[2][2];
            const uint32_t ao = at<C>(i0 + mt * 16 + (lane & 15), ((i0 + kt * 16) >> 3) + (lane >> 4));
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
                put_pair(sm.t[b][0], sm.t[b][1], i0 + mt * 16 + (lane >> 2) + i * 8, j0 + n0 + n * 8 + (lane & 3) * 2,
                         -o[n][2 * i], -o[n][2 * i + 1]);
    }
};

// The chunk's P and T into buffer b from the rows in slot `slot`.  The code is
// kept short (rolled loops): it runs once a chunk beside the other roles', and
// what does not fit the instruction caches is fetched anew each time.
template <int DK, int DVT, bool F32, class S>
__device__ __forceinline__ void prep_chunk(S& sm, int slot, int b, const GdnArgs& a, bool real, int t)
{
    const int warp = t >> 5, lane = t & 31, gq = lane >> 2, q2 = (lane & 3) * 2;
    const uint32_t kb = ptx::smem_u32(sm.k[slot]), qb = ptx::smem_u32(sm.q[slot]);
    const int arow = lane & 15, acol = lane >> 4, brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
    if (warp == 7) scan_rows(sm, b, lane);
    {
        // squared norms of 16 rows of k (warps 0 - 3) or q: the diagonal of their products (bf16 values, exact)
        float d[2][4] = {};
        const uint32_t base = warp < 4 ? kb : qb;
        const int r0 = (warp & 3) * 16;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t x[4], y[4];
            ldsm(x, base + at<DK>(r0 + arow, kt * 2 + acol));
            ldsm(y, base + at<DK>(r0 + brow, kt * 2 + bcol));
            mma_bf(d[0], x, y[0], y[1]);
            mma_bf(d[1], x, y[2], y[3]);
        }
        if (q2 == (gq & 6)) {
            float* n = warp < 4 ? sm.nk : sm.nq;
            n[r0 + gq] = gq & 1 ? d[0][1] : d[0][0];
            n[r0 + gq + 8] = gq & 1 ? d[1][3] : d[1][2];
        }
    }
    prep_sync();
    {
        const int r = t & (C - 1), part = t >> 6;  // halves of k's rows, then of q's
        const float ss = part < 2 ? sm.nk[r] : sm.nq[r];
        float down, up;
        pow2_scale_sqrt(ss, down, up);
        convert_row<DK>(part < 2 ? sm.k[slot] : sm.q[slot], r, part & 1, down);
        // the factor that makes the stored row the (normalised) row; none for a padded one
        const float f = real ? (a.l2 ? rsqrtf(ss + a.l2_eps) : 1.f) * up : 0.f;
        if (part == 0) {
            sm.sk[b][r] = f;
            sm.bk[r] = sm.beta[b][r] * f;
            sm.ek[b][r] = sm.beta[b][r] * f * sm.eg[b][r];
        } else if (part == 2) sm.oq[b][r] = a.scale * f;
    }
    prep_sync();
    // A and P by 16 x 8 tiles on and below the diagonal: twenty over the warps
#pragma unroll 1
    for (int h = warp; h < 20; h += 8) {
        const int blk = h >> 1, bi = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, bj = blk - bi * (bi + 1) / 2;
        const int s0 = bj * 16 + (h & 1) * 8, s = s0 + q2;
        float kk[4] = {}, qk[4] = {};
#pragma unroll
        for (int kp = 0; kp < DK / 32; ++kp) {
            uint32_t ka[2][4], qa[2][4], f[4];
            ldsm(f, kb + at<DK>(s0 + (lane & 7), kp * 4 + (lane >> 3)));
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const uint32_t ao = at<DK>(bi * 16 + arow, kp * 4 + z * 2 + acol);
                ldsm(ka[z], kb + ao);
                ldsm(qa[z], qb + ao);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                mma(kk, ka[z], f[2 * z], f[2 * z + 1]);
                mma(qk, qa[z], f[2 * z], f[2 * z + 1]);
            }
        }
        const float2 ch = *reinterpret_cast<const float2*>(&sm.gh[s]);
        const float2 cl = *reinterpret_cast<const float2*>(&sm.gl[s]);
        const float2 cn = *reinterpret_cast<const float2*>(&sm.sk[b][s]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = bi * 16 + gq + i * 8;
            const float rh = sm.gh[r], rl = sm.gl[r], br = sm.bk[r];
            const float d0 = s <= r ? exp_sfu((rh - ch.x) + (rl - cl.x)) : 0.f;
            const float d1 = s < r ? exp_sfu((rh - ch.y) + (rl - cl.y)) : 0.f;
            const float a0 = s < r ? (br * cn.x) * d0 * kk[2 * i] : 0.f;
            const float a1 = s + 1 < r ? (br * cn.y) * d1 * kk[2 * i + 1] : 0.f;
            const float p0 = s <= r ? d0 * qk[2 * i] : 0.f, p1 = s < r ? d1 * qk[2 * i + 1] : 0.f;
            if (bi == bj) *reinterpret_cast<float2*>(&sm.x[r * XS + (s & 15)]) = make_float2(a0, a1);
            else put_pair(sm.t[b][0], sm.t[b][1], r, s, a0, a1);
            if constexpr (F32) put_pair(sm.p[b][0], sm.p[b][1], r, s, p0, p1);
            else *reinterpret_cast<uint32_t*>(sm.p[b][0] + at<C>(r, s >> 3) + (s & 7) * 2) = pack_h(p0, p1);
        }
    }
    prep_sync();
    if (warp < 4) {
        // a diagonal block for each of four warps: forward substitution, a column a lane
        // (both halves of the warp: one stores the high parts, one the low)
        const int d0 = warp * 16, c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == c ? 1.f : 0.f, acc2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sm.x[(d0 + i) * XS + m]);
                acc = fmaf(-f.x, x[m], acc);
                if (m + 1 < i) acc2 = fmaf(-f.y, x[m + 1], acc2);
                if (m + 2 < i) acc = fmaf(-f.z, x[m + 2], acc);
                if (m + 3 < i) acc2 = fmaf(-f.w, x[m + 3], acc2);
            }
            x[i] = acc + acc2;
        }
        unsigned char* tile = sm.t[b][lane >> 4];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __half hi = __float2half_rn(x[i]);
            const __half lo = __float2half_rn(x[i] - __half2float(hi));
            *reinterpret_cast<__half*>(tile + at<C>(d0 + i, (d0 + c) >> 3) + (c & 7) * 2) = lane < 16 ? hi : lo;
        }
    }
    prep_sync();
    float o[2][4];
    if (warp < 2) {
        const int j0 = warp * 32, i0 = j0 + 16;
        Merge<16> g;
        g.first(sm, b, i0, j0, 0, lane);
        g.second(sm, b, i0, 0, o, lane);
        __syncwarp();
        g.store(sm, b, i0, j0, 0, 0, o, lane);
    }
    prep_sync();
    if (warp < 4) {
        Merge<32> g;
        const int n0 = (warp & 1) * 16, mt = warp >> 1;
        g.first(sm, b, 32, 0, n0, lane);
        g.second(sm, b, 32, mt, o, lane);
        asm volatile("bar.sync 2, 128;" ::: "memory");  // these four warps have read A21
        g.store(sm, b, 32, 0, n0, mt, o, lane);
    }
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

    // S^T K^T, each k-tile's fragments made a tile ahead
    float r[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[t][i] = 0.f;
    __half2 m0 = __float2half2_rn(0.f), m1 = m0;
    uint32_t f[2][4][4], hi[2][4], lo[2][4];
    auto left = [&](int kt) {  // k-tile kt of S^T, split, also for the output warp
#pragma unroll
        for (int t = 0; t < 4; ++t) ldsm(f[kt & 1][t], kb + at<DK>(t * 16 + brow, kt * 2 + bcol));
        uint32_t(&x)[4] = hi[kt & 1], (&y)[4] = lo[kt & 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* v = &s[2 * kt + (i >> 1)][2 * (i & 1)];
            split_h(v[0], v[1], x[i], y[i]);
            const __half2 h = __habs2(*reinterpret_cast<const __half2*>(&x[i]));
            if (i & 1) m1 = __hmax2(m1, h);
            else m0 = __hmax2(m0, h);
        }
        sm.hs[warp][0][kt][lane] = make_uint4(x[0], x[1], x[2], x[3]);
        if (F32) sm.hs[warp][F32 ? 1 : 0][kt][lane] = make_uint4(y[0], y[1], y[2], y[3]);
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
    uint32_t f2[2][4][4];
    auto part = [&](int kt) {
#pragma unroll
        for (int t = kt; t < 4; ++t) {
            ldsm(f[kt & 1][t], tb[0] + at<C>(t * 16 + brow, kt * 2 + bcol));
            ldsm(f2[kt & 1][t], tb[1] + at<C>(t * 16 + brow, kt * 2 + bcol));
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
        uint32_t x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* v = &u[2 * kt + (i >> 1)][2 * (i & 1)];
            if (F32) split_h(v[0] * ud[i & 1], v[1] * ud[i & 1], x[i], y[i]);
            else x[i] = pack_h(v[0] * ud[i & 1], v[1] * ud[i & 1]);
        }
        sm.hu[warp][0][kt][lane] = make_uint4(x[0], x[1], x[2], x[3]);
        if (F32) sm.hu[warp][F32 ? 1 : 0][kt][lane] = make_uint4(y[0], y[1], y[2], y[3]);
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
    auto right = [&](int step) {
#pragma unroll
        for (int t = 0; t < G; ++t)
            ldsm_t(f[step & 1][t], kb + at<DK>(step / NG * 16 + trow, (step % NG * G + t) * 2 + tcol));
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
#pragma unroll 2
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
__global__ void __launch_bounds__(NW * 64 + PREP, 1) gdn_chunk_kernel(const GdnArgs a, const __grid_constant__ RowMaps maps, int dv)
{
    constexpr int DVT = NW * 16, THREADS = NW * 64 + PREP;
    extern __shared__ __align__(1024) unsigned char dyn[];
    using S = Smem<DK, DVT, F32>;
    S& sm = *reinterpret_cast<S*>(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = dv / DVT;
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % a.Hv;
    const int seq = ranked_seq(a.cu_seqlens, a.N, blockIdx.x / (parts * a.Hv), &sm.found);
    int begin, end, slot;
    if (!gdn_unit(a, seq, begin, end, slot)) return;
    const int chunks = (end - begin + C - 1) / C;
    const int col0 = part * DVT;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.ready[i], PREP / 32);
            ptx::mbar_init(&sm.done[i], 2 * NW);
        }
        for (int i = 0; i < 3; ++i) ptx::mbar_init(&sm.loaded[i], 1);
        for (int i = 0; i < NW; ++i) {
            ptx::mbar_init(&sm.s_full[i], 1);
            ptx::mbar_init(&sm.s_free[i], 1);
            ptx::mbar_init(&sm.u_full[i], 1);
            ptx::mbar_init(&sm.u_free[i], 1);
        }
        ptx::fence_mbar_init();
    }
    // T's blocks above the diagonal stay zero
    for (int i = tid; i < (int)sizeof(sm.t) / 16; i += THREADS)
        reinterpret_cast<uint4*>(sm.t)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    Waiter wait{a.dev_status, false};

    // Registers: the launch gives every thread 128 (NW = 4) or 168; the chain
    // warps' warpgroup takes what the others leave.
    if (warp >= 2 * NW) {
        if constexpr (NW == 4) set_regs<false, 104>();
        else set_regs<false, 144>();
        const int t = tid - NW * 64, hk = h / (a.Hv / a.Hk);
        const __nv_bfloat16* ga = static_cast<const __nv_bfloat16*>(a.a) + h;
        const __nv_bfloat16* be = static_cast<const __nv_bfloat16*>(a.b) + h;
        const float ea = expf(a.A_log[h]), dt = a.dt_bias[h];
        __nv_bfloat16 graw = __float2bfloat16(0.f), braw = graw;  // the next chunk's, as loaded
        const uint64_t policy = ptx::policy_evict_normal();  // other heads and columns read the same rows
        auto load = [&](int m) {
            const int r0 = begin + m * C, s = m % 3, r = r0 + (t & (C - 1));
            if (t == PREP - 32) {
                ptx::mbar_arrive_expect_tx(&sm.loaded[s], C * (2 * DK + DVT) * 2);
                load_tile<DK>(sm.k[s], &maps.k, hk * DK, r0, &sm.loaded[s], policy);
                load_tile<DK>(sm.q[s], &maps.q, hk * DK, r0, &sm.loaded[s], policy);
                load_tile<DVT>(sm.v[s], &maps.v, h * dv + col0, r0, &sm.loaded[s], policy);
            }
            if (t < C && r < end) {
                graw = ga[(size_t)r * a.Hv];
                braw = be[(size_t)r * a.Hv];
            }
        };
        load(0);
        for (int m = 0; m < chunks; ++m) {
            const int b = m & 1;
            const bool real = begin + m * C + (t & (C - 1)) < end;
            const float g0 = __bfloat162float(graw), b0 = __bfloat162float(braw);
            if (m >= 2) wait(sm.done[b], (m - 2) >> 1);
            if (t < C) {
                sm.g[t] = real ? gdn_log_alpha(ea, g0, dt) : 0.f;
                sm.beta[b][t] = real ? sigmoidf_(b0) : 0.f;
            }
            if (m + 1 < chunks) load(m + 1);
            wait(sm.loaded[m % 3], m / 3);
            if (begin + m * C + C > end) {
                // the copies took the next sequence's rows along: zeros instead
                const int r = t & (C - 1);
                if (!real && t < C) zero_row<DK>(sm.k[m % 3], r);
                else if (!real && t < 2 * C) zero_row<DK>(sm.q[m % 3], r);
                else if (!real && t < 3 * C) zero_row<DVT>(sm.v[m % 3], r);
            }
            prep_sync();
            prep_chunk<DK, DVT, F32>(sm, m % 3, b, a, real, t);
            ptx::fence_proxy_async_smem();  // the rows written above, before a later copy into their place
            warp_arrive(sm.ready[b], lane);
            prep_sync();  // the scratch and the decays are free again
        }
        return;
    }

    if constexpr (NW == 2) set_regs<true, 208>();
    if (warp >= NW) {
        if constexpr (NW == 4) set_regs<false, 112>();
        const int w = warp - NW;
        const long long row_stride = (long long)a.Hv * dv;
        const size_t osize = F32 ? 4 : 2;
        unsigned char* out = static_cast<unsigned char*>(a.out) + ((size_t)begin * row_stride + (size_t)h * dv + col0) * osize;
        for (int m = 0; m < chunks; ++m) {
            wait(sm.ready[m & 1], m >> 1);
            output_chunk<DK, DVT, F32>(sm, m, out + (size_t)m * C * row_stride * osize, row_stride,
                                       min(C, end - begin - m * C), wait, w, lane);
            ptx::fence_proxy_async_smem();  // outputs staged in the V tile
            warp_arrive(sm.done[m & 1], lane);
        }
        return;
    }

    if constexpr (NW == 4) set_regs<true, 184>();
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
    constexpr int smem = sizeof(Smem<DK, NW * 16, F32>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_chunk_kernel<DK, NW, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    RowMaps maps;
    if (!encode_rows(&maps.q, a.q, (long long)a.Hk * DK, a.qs, a.T, std::min(DK, 64)) ||
        !encode_rows(&maps.k, a.k, (long long)a.Hk * DK, a.ks, a.T, std::min(DK, 64)) ||
        !encode_rows(&maps.v, a.v, (long long)a.Hv * dv, a.vs, a.T, std::min(NW * 16, 64)))
        return cudaErrorInvalidValue;
    gdn_chunk_kernel<DK, NW, F32><<<a.N * a.Hv * (dv / (NW * 16)), NW * 64 + PREP, smem, st>>>(a, maps, dv);
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
