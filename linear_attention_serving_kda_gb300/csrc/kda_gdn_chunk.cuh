// kda_gdn_chunk.cuh -- chunked prefill of the gated delta rule with one decay
// per head (bf16 rows), in chunks of C = 64 rows.
//
// With G the running sum of log alpha in the chunk, row by row:
//     A_rs = beta_r e^{G_r - G_s} k_r.k_s  (s < r),   T = (I + A)^-1
//     R    = diag(beta) V - diag(beta e^G) K S           (U = T R: the rule's updates)
//     S'   = e^{G_C} S + M^T R,   M = T^T diag(e^{G_C - G}) K
//     O    = diag(e^G) Q S + (P T) R,   P_rs = e^{G_r - G_s} q_r.k_s  (s <= r)
// All exponents are differences that are <= 0.  The key rows' factors (powers of two,
// the norm) stay out of T, M and P: with k_r = f_r k'_r, |k'_r| in [1, 2), and F = diag(f),
//     F A F^-1 has the entries beta_r f_r^2 e^{G_r - G_s} k'_r.k'_s,  F R takes R's place,
// and M, P and K S have K' in K's place: no entry of F T F^-1 exceeds 4 while beta |k|^2 <= 2, whatever
// the rows' magnitudes.  Most of the decays stay out of T likewise (D in prep_task: 8 in place of 4).
// Below, A, T, M, P and R are those.
//
// Only S goes from chunk to chunk, so the work is cut where S enters:
//   - prep, a team of eight warps per (chunk, one or two value heads), all chunks at
//     once: K and Q as operands, M and P T, into the workspace;
//   - chains, one CTA per (sequence, value head): R and S' chunk
//     after chunk, two dependent products each, and the outputs beside them.
// The chain is what a long sequence's time is made of; with M in place of T the
// updates U never appear on it.  Up to 64 sequences with work for more than a wave of
// prep run as one grid, chains beside prep (gdn_beside_kernel); others as two kernels one
// after the other.
//
// Bounds and figures (16 key and 32 value heads of 128 x 128, bf16 outputs, 32768 rows).  Dependent
// steps first: prep issues an instruction every other cycle and else waits at its barriers,
// 330 us with 24 warps an SM; a chunk of a chain takes 2.6 us,
// of which the products are 1.0 and the rest the state's way between registers and
// TMEM.  Eight prompts 725 us, one prompt 1350, which is its 512 chunks one after the other.  HBM next:
// rows of 0.8 GB, and a workspace of 1.1 GB written once and read 1.25 times, are 3.3 GB at most, 480 us at the
// copy rate: two thirds of the eight prompts' time, a third of the one's.  The tensor cores are 28 % busy.
// (The beside kernels run at their 80 registers and spill up to 150 bytes of loads a thread.)
//
// Precision: the state keeps fp32 accuracy.  One decay per head leaves k and q
// unscaled inside every product, so the rows' bf16 values are operands without
// loss: prep rescales each row by a power of two to a norm in [1, 2) and stores
// it as fp16 (exact down to 2^-17).  Every other operand
// (S, R, T, M, P, P T) is two fp16 values, high and low, about 22 bits; S and R are
// scaled by a power of two per column and chunk, so that the low part stays in fp16's range.
// That holds for bf16 outputs too: on nearly equal keys an output is a small difference of
// large products, and high parts alone (eight prompts 705 us in place of 725, one 1324 in place
// of 1350) put 3 % of such outputs more than a bf16 step and 1e-3 of their RMS off.
#pragma once

#include <cstddef>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kda_gdn.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int C = 64;
// Float index of 16-byte piece `p` of row r of A's fp32 diagonal blocks: rows of 16 values,
// pieces permuted so that eight rows' same piece lie in distinct banks.
__device__ __forceinline__ int diag_at(int r, int p) { return r * 16 + ((p ^ (r >> 1)) & 3) * 4; }

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
    const float2 d = sub2(make_float2(x, y), unpack_h(hi));
    lo = pack_h(d.x, d.y);
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Byte offsets of 16-byte piece `c` of row `r` in the operand tiles, all with
// 128-byte rows, pieces permuted within eight rows (as a tensor copy with the
// 128-byte swizzle leaves them and the tensor core's descriptors expect them),
// so that eight rows' same piece lie in distinct banks.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return (uint32_t)(r * 128 + (((c ^ r) & 7) << 4)); }
// [K; Q]: 128 rows, 64 values wide, one such tile after the other
__device__ __forceinline__ uint32_t kq_at(int r, int c) { return (uint32_t)((c >> 3) * 16384) + tile_at(r, c); }

// 2^-e and 2^e for the e that brings m into [1, 2), kept within 2^+-60 (so
// that products of two such factors stay finite); 1 for m = 0.
__device__ __forceinline__ void pow2_scale(float m, float& down, float& up)
{
    const uint32_t e = m == 0.f ? 127u : min(max((__float_as_uint(m) >> 23) & 255u, 67u), 187u);
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

// Bounded waits: after one that gives up the others only look once, and the
// role reports it at its end.
struct Waiter {
    bool dead;
    __device__ __forceinline__ void operator()(uint64_t& bar, int phase)
    {
        if (!ptx::mbar_wait_short(&bar, phase & 1, dead ? 1u : 1u << 26)) dead = true;
    }
};

__device__ __forceinline__ void warp_arrive(uint64_t& bar, int lane)
{
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&bar);
}

// ------------------------------------------------------------ workspace

// What prep leaves for a chunk: [K; Q] for each key head, and for each value head
// M^T (dk rows over the chunk's rows) and P T, high and low each, and the factors.
struct Factors {
    float beta[C], ek[C];  // beta f D; beta f^2 e^G D
    float e1[C], e2[C];    // scale, q's row factor, e^G (e1)
    float last;            // e^{G_C}
    float ektop;           // the largest value of ek
    float pad[30];
};
template <int DK> struct Slot {
    static constexpr int HALVES = DK <= 64 ? 1 : DK / 64;  // 64-wide tiles a row spans (dk = 32: half of one)
    static constexpr int KQ = HALVES * 16384, M = DK * 128;
    static constexpr int V = 2 * M + 2 * 8192 + (int)sizeof(Factors);
    static_assert(V % 128 == 0, "slots on the bulk copies' and the operand tiles' boundaries");
};
// A slot is a tile of find_tile: at most T / 64 + N.
__host__ __device__ __forceinline__ long long slot_count(int N, int T) { return (long long)(T / C) + N; }

struct Work {
    unsigned char* kq;  // [slot][Hk]
    unsigned char* v;   // [slot][Hv]
    // where chains run beside prep: [slot][Hv], 1 once the slot is written; then the number of units taken
    int* ready;
    int* taken;
};

// ------------------------------------------------------------ prep

struct RowMaps {
    CUtensorMap q, k, v;
};

constexpr int PREP = 256;
constexpr int PREP_CTAS = 3;  // of an SM, by their shared memory

template <int DK, int HEADS> struct PrepSmem {
    using L = Slot<DK>;
    unsigned char kq[L::KQ];  // bf16 rows of k, then q; fp16 later; P T over q's
    union {
        struct {  // 64 x 64 fp16 tiles
            unsigned char t_hi[8192], t_lo[8192];  // T; then with the rows' factors of M
            unsigned char p_hi[8192], p_lo[8192];
        };
        unsigned char m[2][L::M];  // then M^T
    };
    alignas(16) float xd[C * 16];  // A's diagonal blocks, 16 x 16 each
    // P T: high parts over q's first 64 values, low ones over its last where it has 128, else where P's were
    __device__ __forceinline__ unsigned char* pt_hi() { return kq + 8192; }
    __device__ __forceinline__ unsigned char* pt_lo()
    {
        static_assert(DK == 128 || 2 * L::M <= 16384, "M^T over P's low parts");
        if constexpr (DK == 128) return kq + 16384 + 8192;
        else return p_lo;
    }
    Factors fac[HEADS];
    struct Gates {
        alignas(16) float eg[C], gh[C], gl[C], w[C];  // e^G, G / ln 2 in two words, e^{G_C - G}
    } gates[HEADS];
    alignas(16) float norm[2 * C];  // squared norms of k's and q's rows
    alignas(16) float row[2 * C], col[C];     // factors of A's and P's rows and columns
    alignas(16) float down[2 * C], wd[C];     // of the stored rows; e^{G_C - G} / D
    uint64_t loaded, prod;
    uint32_t tmem;
};

// Barriers of a team of prep warps, and of the four of them that invert T; a CTA has up to three teams.
__device__ __forceinline__ void team_sync(int team) { asm volatile("bar.sync %0, 256;" ::"r"(1 + 2 * team) : "memory"); }
__device__ __forceinline__ void invert_sync(int team) { asm volatile("bar.sync %0, 128;" ::"r"(2 + 2 * team) : "memory"); }

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
template <class S> __device__ __forceinline__ void scan_rows(S& gt, float2 g, float& last, int lane)
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
    *reinterpret_cast<float2*>(&gt.gh[2 * lane]) = make_float2(ph, h);
    *reinterpret_cast<float2*>(&gt.gl[2 * lane]) = make_float2(pl, l);
    *reinterpret_cast<float2*>(&gt.eg[2 * lane]) = make_float2(exp2_sfu(ph + pl), exp2_sfu(h + l));
    *reinterpret_cast<float2*>(&gt.w[2 * lane]) =
        make_float2(exp2_sfu((th - ph) + (tl - pl)), exp2_sfu((th - h) + (tl - l)));
    if (lane == 0) last = exp2_sfu(th + tl);
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
    template <class S> __device__ __forceinline__ void first(S& sm, int i0, int j0, int n0, int lane)
    {
        const uint32_t th = ptx::smem_u32(sm.t_hi), tl = ptx::smem_u32(sm.t_lo);
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
    template <class S> __device__ __forceinline__ void second(S& sm, int i0, int mt, float (&o)[2][4], int lane)
    {
        const uint32_t th = ptx::smem_u32(sm.t_hi), tl = ptx::smem_u32(sm.t_lo);
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
    __device__ __forceinline__ void store(S& sm, int i0, int j0, int n0, int mt, const float (&o)[2][4], int lane)
    {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                put_pair(sm.t_hi, sm.t_lo, i0 + mt * 16 + (lane >> 2) + i * 8, j0 + n0 + n * 8 + (lane & 3) * 2,
                         -o[n][2 * i], -o[n][2 * i + 1]);
    }
};

// One chunk's share of HEADS value heads of one key head by a team of eight
// warps: the rows (r0 .. r0 + n - 1), their products and norms once, then head
// by head.  Bound: latency (a dozen dependent phases of a few hundred
// instructions each); several teams an SM fill each other's gaps.  Task `turn` of
// its team.
template <int DK, int HEADS>
__device__ __forceinline__ void prep_task(PrepSmem<DK, HEADS>& sm, const GdnArgs& a, const RowMaps& maps, const Work& ws,
                                          int slot, int r0, int n, int h0, int turn, int team, uint32_t tmem, Waiter& wait, int t)
{
    using S = PrepSmem<DK, HEADS>;
    using L = Slot<DK>;
    const int w = t >> 5, lane = t & 31, rep = a.Hv / a.Hk, hk = h0 / rep;
    if (t == 0) {
        ptx::mbar_arrive_expect_tx(&sm.loaded, L::KQ);
        const uint64_t policy = ptx::policy_evict_normal();  // the key head's other value heads read the same rows
#pragma unroll 1
        for (int i = 0; i < L::HALVES; ++i) {
            ptx::tma_load_2d(sm.kq + i * 16384, &maps.k, hk * DK + i * 64, r0, &sm.loaded, policy);
            ptx::tma_load_2d(sm.kq + i * 16384 + 8192, &maps.q, hk * DK + i * 64, r0, &sm.loaded, policy);
        }
    }
    // warps 4, 6: a head's gates
    const int gate_head = w == 4 ? 0 : (w == 6 && HEADS == 2) ? 1 : -1;
    float ea = 0.f, dt = 0.f;
    if (gate_head >= 0) {
        ea = a.A_log[h0 + gate_head];
        dt = a.dt_bias[h0 + gate_head];
    }
    float graw[2] = {0.f, 0.f}, braw[2] = {0.f, 0.f};
    if (gate_head >= 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < n) {
                const size_t at = (size_t)(r0 + 2 * lane + i) * a.Hv + h0 + gate_head;
                graw[i] = ldv(static_cast<const __nv_bfloat16*>(a.a) + at);
                braw[i] = ldv(static_cast<const __nv_bfloat16*>(a.b) + at);
            }
    }
    if (w == 0) {
        wait(sm.loaded, turn);
        if (lane == 0) {
            // [K; Q] [K; Q]^T: k.k, q.k and, on the diagonal, both squared norms
            ptx::tc_fence_after();  // the team has read the task before this one
            const uint32_t kq = ptx::smem_u32(sm.kq);
#pragma unroll
            for (int kt = 0; kt < DK / 16; ++kt) {
                const uint64_t d = ptx::desc_sw128(kq + (kt >> 2) * 16384 + (kt & 3) * 32);
                ptx::mma_f16_ss(tmem, d, d, ptx::idesc_bf16(128, 128), kt > 0);
            }
            ptx::mma_commit(&sm.prod);
        }
        __syncwarp();
    }
    if (gate_head >= 0) {
        // two rows a lane; a padded row decays nothing and takes nothing
        ea = expf(ea) * 1.44269504088896341f;
        float g[2] = {0.f, 0.f}, bt[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < n) {
                g[i] = gdn_log_alpha(ea, graw[i], dt);
                bt[i] = sigmoidf_(braw[i]);
            }
        sm.fac[gate_head].beta[2 * lane] = bt[0];
        sm.fac[gate_head].beta[2 * lane + 1] = bt[1];
        if (lane == 0) sm.fac[gate_head].ektop = 0.f;
        scan_rows(sm.gates[gate_head], make_float2(g[0], g[1]), sm.fac[gate_head].last, lane);
    }
    // a row of [K; Q] a lane (w & 3), against half of k's rows (w >> 2); the
    // halves above the diagonal (w = 4 and 6) are left out
    const int lr = (w & 3) * 32 + lane, r = lr & (C - 1), type = lr >> 6, s0 = (w >> 2) * 32;  // type 0: k, 1: q
    const uint32_t at = tmem + ((uint32_t)((w & 3) * 32) << 16);
    wait(sm.prod, turn);
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
    team_sync(team);
    const int arow = lane & 15, acol = lane >> 4, brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
    auto store_tile = [&](unsigned char* hi_tile, unsigned char* lo_tile, int row0, const float (&c)[8][4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_h(c[2 * q + (i >> 1)][2 * (i & 1)], c[2 * q + (i >> 1)][2 * (i & 1) + 1], hi[i], lo[i]);
            const uint32_t o = tile_at(row0 + arow, q * 2 + acol);
            stsm(ptx::smem_u32(hi_tile) + o, hi);
            stsm(ptx::smem_u32(lo_tile) + o, lo);
        }
    };

#pragma unroll 1
    for (int j = 0; j < HEADS; ++j) {
        const typename S::Gates& gt = sm.gates[j];
        Factors& fac = sm.fac[j];
        if (w < 4) {
            const float ss = sm.norm[lr];
            float down, up;
            pow2_scale_sqrt(ss, down, up);
            // f: what makes the stored row the (normalised) row; none for a padded one
            const float nrm = r < n ? (a.l2 ? rsqrtf(ss + a.l2_eps) : 1.f) : 0.f, f = nrm * up;
            sm.down[lr] = down;
            if (type == 0) {
                // D R takes R's place, D a power of two near e^{G_C - G}, so that rows which the chunk's end
                // has forgotten do not set the scale of those it has not; and D T D^-1, M D^-1 and P D^-1 those
                // of T, M and P: with T's decays left in it, its small entries (and what M made of them, divided by D)
                // would be at fp16's smallest step.  D >= 2^-12 for P's sake (its entries stay below 2^14)
                const float dd = __uint_as_float(__float_as_uint(fminf(fmaxf(gt.w[r], 0x1p-12f), 1.f)) & 0x7f800000u);
                const float be = fac.beta[r] * dd, ek = be * f * f * gt.eg[r];
                const float inv = __uint_as_float((254u << 23) - __float_as_uint(dd));
                sm.col[r] = down * inv;
                sm.wd[r] = gt.w[r] * inv;
                fac.beta[r] = be * f;
                fac.ek[r] = ek;
                atomicMax(reinterpret_cast<int*>(&fac.ektop), __float_as_int(fabsf(ek)));  // >= 0: ordered as integers
                sm.row[r] = be * nrm * f;  // from the raw rows' products, with their columns' down
            } else {
                fac.e1[r] = a.scale * f * gt.eg[r];
                fac.e2[r] = a.scale * f;
                sm.row[lr] = down;
            }
        }
        if (j > 0 && t == 0) ptx::bulk_wait_read_all();  // the head before this one has left the tiles
        team_sync(team);
        if (w != 4 && w != 6) {
            // the lane's row of A (beta_r |..| e^{G_r - G_s} k_r.k_s) or P, zero from the diagonal (or past it) on
            const float rh = gt.gh[r], rl = gt.gl[r], rf = sm.row[lr];
            const int lim = r < n ? r + type : 0;
            unsigned char* hi_tile = type == 0 ? sm.t_hi : sm.p_hi;
            unsigned char* lo_tile = type == 0 ? sm.t_lo : sm.p_lo;
#pragma unroll 2
            for (int p = 0; p < 4; ++p) {
                uint32_t hi[4], lo[4];
                float v[8], d[8];
                ptx::tmem_ld8(at + s0 + p * 8, d);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int s = s0 + p * 8 + z * 2;
                    const float2 ch = *reinterpret_cast<const float2*>(&gt.gh[s]);
                    const float2 cl = *reinterpret_cast<const float2*>(&gt.gl[s]);
                    const float2 c2 = *reinterpret_cast<const float2*>(&sm.col[s]);
                    const float2 e = add2(sub2(both2(rh), ch), sub2(both2(rl), cl));
                    // (rf c2 may be infinite, of rows of zeros say)
                    const float2 x = mul2(mul2(both2(rf), make_float2(exp2_sfu(e.x), exp2_sfu(e.y))),
                                          mul2(c2, make_float2(d[2 * z], d[2 * z + 1])));
                    v[2 * z] = s < lim ? x.x : 0.f;
                    v[2 * z + 1] = s + 1 < lim ? x.y : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) split_h(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
                const int c = (s0 >> 3) + p;
                *reinterpret_cast<uint4*>(hi_tile + tile_at(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(lo_tile + tile_at(r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (type == 0 && (r >> 4) == (c >> 1)) {
                    *reinterpret_cast<float4*>(&sm.xd[diag_at(r, (c & 1) * 2)]) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4*>(&sm.xd[diag_at(r, (c & 1) * 2 + 1)]) = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
        }
        ptx::tc_fence_before();
        team_sync(team);
        if (w >= 4) {
            // meanwhile the rows themselves
            if (j == 0) {
                const int row = (w - 4) * 32 + lane;
                wait(sm.loaded, turn);
                convert_row<DK>(sm.kq, row, sm.down[row], (row & (C - 1)) < n);
                ptx::fence_proxy_async_smem();
            }
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
                    for (int k = 0; k < i; k += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&sm.xd[diag_at(d0 + i, k >> 2)]);
                        acc = fmaf(-f.x, x[k], acc);
                        if (k + 1 < i) acc2 = fmaf(-f.y, x[k + 1], acc2);
                        if (k + 2 < i) acc = fmaf(-f.z, x[k + 2], acc);
                        if (k + 3 < i) acc2 = fmaf(-f.w, x[k + 3], acc2);
                    }
                    x[i] = acc + acc2;
                }
                unsigned char* tile = lane < 16 ? sm.t_hi : sm.t_lo;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const __half hi = __float2half_rn(x[i]);
                    const __half lo = __float2half_rn(x[i] - __half2float(hi));
                    *reinterpret_cast<__half*>(tile + tile_at(d0 + i, (d0 + c) >> 3) + (c & 7) * 2) = lane < 16 ? hi : lo;
                }
            }
            invert_sync(team);
            float o[2][4];
            if (w < 2) {
                const int j0 = w * 32, i0 = j0 + 16;
                Merge<16> mg;
                mg.first(sm, i0, j0, 0, lane);
                mg.second(sm, i0, 0, o, lane);
                __syncwarp();
                mg.store(sm, i0, j0, 0, 0, o, lane);
            }
            invert_sync(team);
            Merge<32> mg;
            const int n0 = (w & 1) * 16, mt = w >> 1;
            mg.first(sm, 32, 0, n0, lane);
            mg.second(sm, 32, mt, o, lane);
            invert_sync(team);  // every warp has read A21
            mg.store(sm, 32, 0, n0, mt, o, lane);
        }
        team_sync(team);
        if (j == 0 && t == 0 && h0 % rep == 0) {
            ptx::bulk_s2g(ws.kq + ((long long)slot * a.Hk + hk) * L::KQ, sm.kq, L::KQ);
            ptx::bulk_commit();
        }
        float c[8][4];
        auto clear = [&] {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
        };
        clear();
        if (w >= 4) {
            // P T: sixteen rows a warp
            const int mt = w - 4;
            const uint32_t pb[2] = {ptx::smem_u32(sm.p_hi), ptx::smem_u32(sm.p_lo)};
            const uint32_t tb[2] = {ptx::smem_u32(sm.t_hi), ptx::smem_u32(sm.t_lo)};
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                if (kt > mt) break;  // P's columns up to its rows
                uint32_t x[4], y[4], f[4], e[4];
                ldsm(x, pb[0] + tile_at(mt * 16 + arow, kt * 2 + acol));
                ldsm(y, pb[1] + tile_at(mt * 16 + arow, kt * 2 + acol));
#pragma unroll
                for (int q = 0; q <= kt; ++q) {
                    ldsm_t(f, tb[0] + tile_at(kt * 16 + arow, q * 2 + acol));
                    mma(c[2 * q], x, f[0], f[1]);
                    mma(c[2 * q + 1], x, f[2], f[3]);
                    ldsm_t(e, tb[1] + tile_at(kt * 16 + arow, q * 2 + acol));
                    mma(c[2 * q], y, f[0], f[1]);
                    mma(c[2 * q + 1], y, f[2], f[3]);
                    mma(c[2 * q], x, e[0], e[1]);
                    mma(c[2 * q + 1], x, e[2], e[3]);
                }
            }
        } else if (t == 0) ptx::bulk_wait_read_all();  // [K; Q] is on its way: room for P T over q's rows
        team_sync(team);
        if (w >= 4) store_tile(sm.pt_hi(), sm.pt_lo(), (w - 4) * 16, c);
        // T with M's row factors, in pieces of eight values up to each diagonal block's end: 32 + 64 + 96 + 128
#pragma unroll 1
        for (int i = t; i < 320; i += PREP) {
            const int kt = i < 32 ? 0 : i < 96 ? 1 : i < 192 ? 2 : 3, l = i - 16 * kt * (kt + 1);
            const int rr = kt * 16 + l / (2 * kt + 2), pc = l % (2 * kt + 2);
            const float f = sm.wd[rr];
            uint4* hp = reinterpret_cast<uint4*>(sm.t_hi + tile_at(rr, pc));
            uint4* lp = reinterpret_cast<uint4*>(sm.t_lo + tile_at(rr, pc));
            const uint4 h4 = *hp, l4 = *lp;
            const uint32_t hv[4] = {h4.x, h4.y, h4.z, h4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
            uint32_t wh[4], wl[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float2 x = mul2(add2(unpack_h(hv[z]), unpack_h(lv[z])), both2(f));
                split_h(x.x, x.y, wh[z], wl[z]);
            }
            *hp = make_uint4(wh[0], wh[1], wh[2], wh[3]);
            *lp = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        }
        team_sync(team);
        clear();
        if (w * 16 < DK) {
            // M^T: sixteen of dk's rows a warp, K'^T (exact) times T's high and low; row r of T meets columns s <= r
            const uint32_t kb = ptx::smem_u32(sm.kq), th = ptx::smem_u32(sm.t_hi), tl = ptx::smem_u32(sm.t_lo);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint32_t x[4], f[4], e[4];
                // left operand (dk, r) from rows r of k: transposed
                ldsm_t(x, kb + kq_at(kt * 16 + brow, w * 2 + bcol));
#pragma unroll
                for (int q = 0; q <= kt; ++q) {
                    ldsm_t(f, th + tile_at(kt * 16 + arow, q * 2 + acol));
                    ldsm_t(e, tl + tile_at(kt * 16 + arow, q * 2 + acol));
                    mma(c[2 * q], x, f[0], f[1]);
                    mma(c[2 * q + 1], x, f[2], f[3]);
                    mma(c[2 * q], x, e[0], e[1]);
                    mma(c[2 * q + 1], x, e[2], e[3]);
                }
            }
        }
        team_sync(team);  // the tiles read above make room
        if (w * 16 < DK) store_tile(sm.m[0], sm.m[1], w * 16, c);
        ptx::fence_proxy_async_smem();
        team_sync(team);
        if (t == 0) {
            unsigned char* d = ws.v + ((long long)slot * a.Hv + h0 + j) * L::V;
            ptx::bulk_s2g(d, sm.m, 2 * L::M);
            ptx::bulk_s2g(d + 2 * L::M, sm.pt_hi(), 8192);
            ptx::bulk_s2g(d + 2 * L::M + 8192, sm.pt_lo(), 8192);
            ptx::bulk_s2g(d + 2 * L::M + 2 * 8192, &fac, sizeof(Factors));
            ptx::bulk_commit();
        }
    }
}

template <int DK, int HEADS> __device__ __forceinline__ void prep_setup(PrepSmem<DK, HEADS>& sm, int t)
{
    if (t == 0) {
        ptx::mbar_init(&sm.loaded, 1);
        ptx::mbar_init(&sm.prod, 1);
        ptx::fence_mbar_init();
    }
}

// A task a CTA.
template <int DK, int HEADS>
__global__ void __launch_bounds__(PREP, PREP_CTAS)
gdn_prep_kernel(const GdnArgs a, const __grid_constant__ RowMaps maps, const Work ws)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    extern __shared__ __align__(1024) unsigned char dyn[];
    using S = PrepSmem<DK, HEADS>;
    S& sm = *reinterpret_cast<S*>(dyn);
    const int t = threadIdx.x, lane = t & 31, groups = a.Hv / HEADS, slot = blockIdx.x / groups;
    // every warp for itself: the rows of this slot
    int begin, end;
    const int seq = find_tile<C>(a.cu_seqlens, a.N, a.T, slot, lane, begin, end);
    if (seq < 0) return;
    const int r0 = begin + (slot - begin / C - seq) * C, n = min(C, end - r0);
    prep_setup(sm, t);
    if (t / 32 == 1) ptx::tmem_alloc(&sm.tmem, 128);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    Waiter wait{false};
    prep_task<DK, HEADS>(sm, a, maps, ws, slot, r0, n, blockIdx.x % groups * HEADS, 0, 0, sm.tmem, wait, t);
    if (wait.dead) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
    if (t == 0) ptx::bulk_wait_read_all();
    if (t / 32 == 1) ptx::tmem_dealloc(sm.tmem, 128);
}

// ------------------------------------------------------------ chain

// TMEM columns: the critical products (K S; then M^T R), S high and low, R high
// and low as left operands (two fp16 a column), Q S, (P T) R
// (the first of them as two halves, K S high and K S low)
constexpr int TM_X = 0, TM_SH = 128, TM_SL = 192, TM_RH = 256, TM_RL = 288, TM_QS = 320, TM_PR = 384, TM_COLS = 512;
constexpr int CHAIN_THREADS = 640;

// A sequence's rows, its state and value head.
struct Unit {
    int seq, begin, end, slot, h;
};

template <int DK, int DV> struct ChainSmem {
    using L = Slot<DK>;
    unsigned char kq[2][L::KQ];
    unsigned char work[2][2 * L::M + 2 * 8192];       // M^T, P T
    unsigned char v[2][C * DV * 2];                     // dense rows
    Factors fac[4];
    float f1[2][DV], f2[2][DV];  // the scales of S's and R's columns
    float top[2][2][DV];         // the largest values of beta V's and S's halves of a column
    uint64_t loaded[2], freed[2];
    uint64_t s_full, ks_full, qs_full, rh_full, rl_full, su_full, o_full, o_free, f_full[2];
    int found;
    Unit unit;
};

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }

// Values two by two as fp16 high parts and what those leave as low parts, N / 2
// columns each.
template <int N> __device__ __forceinline__ void store_pairs(uint32_t at, const uint32_t (&v)[N])
{
    static_assert(N == 8 || N % 16 == 0, "columns");
    if constexpr (N == 8) ptx::tmem_st8(at, v);
    else {
#pragma unroll
        for (int b = 0; b < N; b += 16) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = v[b + i];
            ptx::tmem_st16_async(at + b, w);
        }
    }
}
template <int N> __device__ __forceinline__ void scale_all(float (&x)[N], float f)
{
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 y = mul2(make_float2(x[i], x[i + 1]), both2(f));
        x[i] = y.x;
        x[i + 1] = y.y;
    }
}
template <int N> __device__ __forceinline__ void store_high(uint32_t at, const float (&x)[N])
{
    uint32_t v[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = pack_h(x[2 * i], x[2 * i + 1]);
    store_pairs(at, v);
    ptx::tmem_wait_st();
}
template <int N> __device__ __forceinline__ void store_low(uint32_t at, const float (&x)[N])
{
    uint32_t v[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        uint32_t hi;
        split_h(x[2 * i], x[2 * i + 1], hi, v[i]);
    }
    store_pairs(at, v);
    ptx::tmem_wait_st();
}
template <int N> __device__ __forceinline__ void store_split(uint32_t hi_at, uint32_t lo_at, const float (&x)[N])
{
    constexpr int B = N < 32 ? N : 32;
#pragma unroll
    for (int b = 0; b < N; b += B) {
        uint32_t hi[B / 2], lo[B / 2];
#pragma unroll
        for (int i = 0; i < B / 2; ++i) split_h(x[b + 2 * i], x[b + 2 * i + 1], hi[i], lo[i]);
        store_pairs(hi_at + b / 2, hi);
        store_pairs(lo_at + b / 2, lo);
    }
    ptx::tmem_wait_st();
}

// Sets the register count of the calling warpgroup's threads.
template <bool UP, int N> __device__ __forceinline__ void set_regs()
{
    if constexpr (UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The chain's 640 threads.
__device__ __forceinline__ void chain_sync() { asm volatile("bar.sync 7, 640;" ::: "memory"); }

// What a CTA's chain units are.  One for each CTA:
struct OneUnit {
    static constexpr bool BESIDE = false;
    Unit u;
    template <class S> __device__ __forceinline__ bool next(S&, const GdnArgs&, const Work&, int turn, Unit& out)
    {
        out = u;
        return turn == 0;
    }
};

// The chains of one unit after the other.  The barriers' phases, the buffers
// and TMEM go on from unit to unit: only `q`, the chunk's number among all of the
// CTA's, counts for them.  tmem: all of it; freed here.
template <int DK, int DV, bool OUT32, class Units>
__device__ __forceinline__ void run_chains(unsigned char* dyn, const GdnArgs& a, const CUtensorMap& vmap, const Work& ws, uint32_t tmem, Units units)
{
    constexpr int NW = DV / 32;
    using S = ChainSmem<DK, DV>;
    using L = Slot<DK>;
    S& sm = *reinterpret_cast<S*>(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.loaded[i], 1);
            ptx::mbar_init(&sm.freed[i], 2 * NW + 1);
            ptx::mbar_init(&sm.f_full[i], NW);
        }
        ptx::mbar_init(&sm.s_full, 2 * NW);
        ptx::mbar_init(&sm.ks_full, 2);
        ptx::mbar_init(&sm.qs_full, 1);
        ptx::mbar_init(&sm.rh_full, 2 * NW);
        ptx::mbar_init(&sm.rl_full, 2 * NW);
        ptx::mbar_init(&sm.su_full, 1);
        ptx::mbar_init(&sm.o_full, 1);
        ptx::mbar_init(&sm.o_free, 2 * NW);
        ptx::fence_mbar_init();
    }
    chain_sync();
    Waiter wait{false};
    Unit u;
    int q0 = 0;  // chunks of the units before

    // Registers: the launch gives every thread 96 (beside prep: 80, and there is a
    // sixth warpgroup); the chain's two warpgroups take what the others leave
    // (2 * 144 + 3 * 64 = 5 * 96; 2 * 144 + 3 * 56 + 24 = 6 * 80).
    constexpr int FEW = Units::BESIDE ? 56 : 64;
    if (warp < 8) {
        set_regs<true, 144>();
        if ((warp & 3) < NW) {
            // column c of the state, scaled by g; of each product's columns (dk, then
            // the chunk's rows) this warp has one half, its partner the other
            constexpr int SK = DK / 2, RK = C / 2;
            const int pair = warp & 3, half = warp >> 2, c = pair * 32 + lane;
            const uint32_t at = tmem + ((uint32_t)(pair * 32) << 16);
            // the larger of both halves' largest values (each in its place by now)
            auto both = [&](int which, float x) {
                asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
                return fmaxf(x, sm.top[which][half ^ 1][c]);
            };
            for (int turn = 0; units.next(sm, a, ws, turn, u); ++turn) {
                const int begin = u.begin, end = u.end, chunks = (end - begin + C - 1) / C;
                float* state = a.state + ((size_t)u.slot * a.Hv + u.h) * DK * DV + (size_t)half * SK * DV + c;
                // s is S times g, the power of two of the column that brings its largest
                // value near one for the fp16 operands.  Decays of many orders of magnitude a chunk are
                // ordinary, and a value that has become much smaller than one would lose digits of its low part:
                // so every chunk looks at the largest value again, and changes g where it is off.
                float s[SK], g = 1.f, ig = 1.f;
#pragma unroll
                for (int i = 0; i < SK; ++i) s[i] = state[(size_t)i * DV];
                for (int m = 0; m < chunks; ++m) {
                    const int q = q0 + m, b = q & 1, n = end - begin - m * C;
                    if (q > 0) wait(sm.qs_full, q - 1);  // S's place is free
                    float most = 0.f, mx = 0.f;
#pragma unroll
                    for (int i = 0; i < SK; i += 2) most = max3(most, fabsf(s[i]), fabsf(s[i + 1]));
                    // stored before the other half's largest value is known, and again where g was off
                    sm.top[1][half][c] = most;
                    store_split<SK>(at + TM_SH + half * (SK / 2), at + TM_SL + half * (SK / 2), s);
                    most = both(1, most);
                    const bool off = !(most >= 0.125f && most < 0x1p14f) && most != 0.f;
                    if (__any_sync(0xffffffffu, off)) {
                        float down, up;
                        pow2_scale(off ? most * ig : ig, down, up);
                        const float f = down * ig;
                        scale_all(s, f);
                        most *= f;
                        g = down;
                        ig = up;
                        store_split<SK>(at + TM_SH + half * (SK / 2), at + TM_SL + half * (SK / 2), s);
                    }
                    ptx::tc_fence_before();
                    warp_arrive(sm.s_full, lane);

                    // R = beta V - beta e^G k.S, times rd
                    wait(sm.loaded[b], q >> 1);
                    const Factors& fac = sm.fac[q & 3];
                    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(sm.v[b]) + half * RK * DV + c;
                    float r[RK];
#pragma unroll
                    for (int i = 0; i < RK; i += 2) {
                        const float2 be = *reinterpret_cast<const float2*>(&fac.beta[half * RK + i]);
                        const float2 x = mul2(be, make_float2(__bfloat162float(v[i * DV]), __bfloat162float(v[(i + 1) * DV])));
                        r[i] = x.x;
                        r[i + 1] = x.y;
                    }
                    if (n < C)  // the copies took the next sequence's rows along
#pragma unroll
                        for (int i = 0; i < RK; ++i) r[i] = half * RK + i < n ? r[i] : 0.f;
#pragma unroll
                    for (int i = 0; i < RK; i += 2) mx = max3(mx, fabsf(r[i]), fabsf(r[i + 1]));
                    sm.top[0][half][c] = mx;
                    // |k'| < 2, so |k'.S| <= 2 sqrt(dk) max |S|: R stays below 2^14 in the scale of this
                    // bound, and low parts do not mind how far below; 2^-60 of S at least, so that ig rd is finite
                    float rd, ru;
                    pow2_scale(fmaxf(both(0, mx) + fac.ektop * (DK == 128 ? 23.f : DK == 64 ? 16.f : 12.f) * (most * ig),
                                     0x1p-60f * (most * ig)), rd, ru);
                    rd *= 0x1p13f;
                    ru *= 0x1p-13f;
                    scale_all(r, rd);
                    if (q > 0) wait(sm.o_full, q - 1);  // R's place is free
                    wait(sm.ks_full, q);
                    ptx::tc_fence_after();
                    const float fr = most == 0.f ? 0.f : ig * rd;  // an S of zeros may have any ig
#pragma unroll
                    for (int z = 0; z < RK; z += 16) {
                        float d[16], e[16];
                        ptx::tmem_ld16(at + TM_X + half * RK + z, d);
                        ptx::tmem_ld16(at + TM_X + C + half * RK + z, e);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 ek = *reinterpret_cast<const float2*>(&fac.ek[half * RK + z + i]);
                            const float2 ks = mul2(add2(make_float2(d[i], d[i + 1]), make_float2(e[i], e[i + 1])), both2(-fr));
                            const float2 x = fma2(ek, ks, make_float2(r[z + i], r[z + i + 1]));
                            r[z + i] = x.x;
                            r[z + i + 1] = x.y;
                        }
                    }
                    store_high<RK>(at + TM_RH + half * (RK / 2), r);
                    ptx::tc_fence_before();
                    warp_arrive(sm.rh_full, lane);
                    store_low<RK>(at + TM_RL + half * (RK / 2), r);
                    ptx::tc_fence_before();
                    warp_arrive(sm.rl_full, lane);
                    if (half == 0) {
                        sm.f1[b][c] = ig;
                        sm.f2[b][c] = ru;
                        warp_arrive(sm.f_full[b], lane);
                    }

                    // S = e^{G_C} S + M^T R
                    scale_all(s, fac.last);
                    const float fs = ru * g;
                    wait(sm.su_full, q);
                    ptx::tc_fence_after();
                    constexpr int W = SK < 32 ? SK : 32;
#pragma unroll
                    for (int z = 0; z < SK; z += W) {
                        float d[W];
                        if constexpr (W == 32) ptx::tmem_ld32(at + TM_X + half * SK + z, d);
                        else ptx::tmem_ld16(at + TM_X + half * SK + z, d);
#pragma unroll
                        for (int i = 0; i < W; i += 2) {
                            const float2 x = fma2(both2(fs), make_float2(d[i], d[i + 1]), make_float2(s[z + i], s[z + i + 1]));
                            s[z + i] = x.x;
                            s[z + i + 1] = x.y;
                        }
                    }
                    warp_arrive(sm.freed[b], lane);
                }
#pragma unroll
                for (int i = 0; i < SK; ++i) state[(size_t)i * DV] = s[i] * ig;
                q0 += chunks;
            }
        } else
            for (int turn = 0; units.next(sm, a, ws, turn, u);) ++turn;
    } else if (warp < 12) {
        set_regs<false, FEW>();
        auto kq_step = [](int kt) { return (uint64_t)((kt >> 2) * (16384 >> 4) + (kt & 3) * 2); };
        constexpr uint32_t id = ptx::idesc_f16(128, C), idm = ptx::idesc_f16(128, DK);
        if (warp == 8) {
            const uint64_t policy = ptx::policy_evict_first();
            for (int turn = 0; units.next(sm, a, ws, turn, u); ++turn) {
                const int begin = u.begin, end = u.end, chunks = (end - begin + C - 1) / C;
                const int h = u.h;
                const long long slot0 = begin / C + u.seq;
                for (int m = 0; m < chunks; ++m) {
                    const int q = q0 + m, b = q & 1;
                    // a chunk's operands are free once its products are through; its factors
                    // are read a little longer, while its outputs are formed: a ring of four
                    if (q >= 2) wait(sm.freed[b], (q - 2) >> 1);
                    if (Units::BESIDE) {
                        // this head's slot, and that of the key head's first, which brings [K; Q]
                        const int* f = ws.ready + (slot0 + m) * a.Hv;
                        const int lead = h / (a.Hv / a.Hk) * (a.Hv / a.Hk);
                        if (!wait.dead && !(ptx::wait_flag_ge(f + lead, 1) && ptx::wait_flag_ge(f + h, 1))) wait.dead = true;
                        ptx::fence_proxy_async_global();
                    }
                    if (lane == 0) {
                        uint64_t* bar = &sm.loaded[b];
                        const unsigned char* w = ws.v + ((slot0 + m) * a.Hv + h) * L::V;
                        ptx::mbar_arrive_expect_tx(bar, L::KQ + L::V + C * DV * 2);
                        ptx::bulk_g2s(sm.kq[b], ws.kq + ((slot0 + m) * a.Hk + h / (a.Hv / a.Hk)) * L::KQ, L::KQ, bar);
                        ptx::tma_load_2d(sm.v[b], &vmap, h * DV, begin + m * C, bar, policy);
                        ptx::bulk_g2s_stream(&sm.fac[q & 3], w + sizeof(sm.work[0]), sizeof(Factors), bar, policy);
                        ptx::bulk_g2s_stream(sm.work[b], w, sizeof(sm.work[0]), bar, policy);
                    }
                    __syncwarp();
                }
                q0 += chunks;
            }
        } else if (warp == 9 || warp == 10) {
            // The critical products from two warps: K S of S's high parts and M^T R, K S of
            // its low parts.  The warps stay whole and one lane of each issues: from a branch of
            // that lane's own every operand is moved over first, and a long prompt
            // takes 5 % longer.
            const bool first = warp == 9;
            const uint32_t leader = ptx::elect_one();
            for (int turn = 0; units.next(sm, a, ws, turn, u); ++turn) {
                const int chunks = __shfl_sync(0xffffffffu, (u.end - u.begin + C - 1) / C, 0);
                for (int m = 0; m < chunks; ++m) {
                    const int q = q0 + m, b = q & 1;
                    wait(sm.loaded[b], q >> 1);
                    wait(sm.s_full, q);
                    __syncwarp();
                    ptx::tc_fence_after();
                    const uint64_t k = ptx::desc_sw128(ptx::smem_u32(sm.kq[b]));
                    const uint64_t mh = ptx::desc_sw128(ptx::smem_u32(sm.work[b])), ml = mh + (L::M >> 4);
                    const uint32_t d = tmem + TM_X + (first ? 0 : C), s = tmem + (first ? TM_SH : TM_SL);
#pragma unroll
                    for (int kt = 0; kt < DK / 16; ++kt) ptx::mma_ts_if(leader, d, s + kt * 8, k + kq_step(kt), id, kt > 0);
                    ptx::mma_commit_if(leader, &sm.ks_full);
                    __syncwarp();
                    if (!first) continue;
                    wait(sm.rh_full, q);
                    __syncwarp();
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_X, tmem + TM_RH + kt * 8, mh + kt * 2, idm, kt > 0);
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_X, tmem + TM_RH + kt * 8, ml + kt * 2, idm, 1);
                    __syncwarp();
                    wait(sm.rl_full, q);
                    __syncwarp();
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_X, tmem + TM_RL + kt * 8, mh + kt * 2, idm, 1);
                    ptx::mma_commit_if(leader, &sm.su_full);
                    __syncwarp();
                }
                q0 += chunks;
            }
        } else {
            // the outputs' products, each behind the critical ones of its kind
            const uint32_t leader = ptx::elect_one();
            for (int turn = 0; units.next(sm, a, ws, turn, u); ++turn) {
                const int chunks = __shfl_sync(0xffffffffu, (u.end - u.begin + C - 1) / C, 0);
                for (int m = 0; m < chunks; ++m) {
                    const int q = q0 + m, b = q & 1;
                    if (q > 0) wait(sm.o_free, q - 1);
                    wait(sm.loaded[b], q >> 1);
                    wait(sm.ks_full, q);
                    __syncwarp();
                    ptx::tc_fence_after();
                    const uint64_t qd = ptx::desc_sw128(ptx::smem_u32(sm.kq[b]) + 8192);
                    const uint64_t pt = ptx::desc_sw128(ptx::smem_u32(sm.work[b]) + 2 * L::M);
#pragma unroll
                    for (int kt = 0; kt < DK / 16; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_QS, tmem + TM_SH + kt * 8, qd + kq_step(kt), id, kt > 0);
#pragma unroll
                    for (int kt = 0; kt < DK / 16; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_QS, tmem + TM_SL + kt * 8, qd + kq_step(kt), id, 1);
                    ptx::mma_commit_if(leader, &sm.qs_full);
                    __syncwarp();
                    wait(sm.su_full, q);
                    __syncwarp();
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        ptx::mma_ts_if(leader, tmem + TM_PR, tmem + TM_RH + kt * 8, pt + kt * 2, id, kt > 0);
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt) {
                        ptx::mma_ts_if(leader, tmem + TM_PR, tmem + TM_RL + kt * 8, pt + kt * 2, id, 1);
                        ptx::mma_ts_if(leader, tmem + TM_PR, tmem + TM_RH + kt * 8, pt + (8192 >> 4) + kt * 2, id, 1);
                    }
                    ptx::mma_commit_if(leader, &sm.freed[b]);
                    ptx::mma_commit_if(leader, &sm.o_full);
                    __syncwarp();
                }
                q0 += chunks;
            }
        }
    } else {
        set_regs<false, FEW>();
        if ((warp & 3) < NW) {
            // column c of the outputs: o_r = e1 q'.S + e2 (P T R)_r, for half of the rows
            const int w = warp & 3, c = w * 32 + lane, half = (warp - 12) >> 2;
            const uint32_t at = tmem + ((uint32_t)(w * 32) << 16);
            const size_t row_stride = (size_t)a.Hv * DV;
            for (int turn = 0; units.next(sm, a, ws, turn, u); ++turn) {
                const int begin = u.begin, end = u.end, chunks = (end - begin + C - 1) / C;
                for (int m = 0; m < chunks; ++m) {
                    const int q = q0 + m, b = q & 1, n = min(C, end - begin - m * C);
                    wait(sm.f_full[b], q >> 1);
                    const float f1 = sm.f1[b][c], f2 = sm.f2[b][c];
                    const Factors& fac = sm.fac[q & 3];
                    const size_t o0 = ((size_t)begin + (size_t)m * C) * row_stride + (size_t)u.h * DV;
                    wait(sm.o_full, q);
                    ptx::tc_fence_after();
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int i0 = half * (C / 2) + z * 16;
                        float x[16], y[16];
                        ptx::tmem_ld16(at + TM_QS + i0, x);
                        ptx::tmem_ld16(at + TM_PR + i0, y);
                        if (z == 1) {
                            ptx::tc_fence_before();
                            warp_arrive(sm.o_free, lane);
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 e1 = *reinterpret_cast<const float2*>(&fac.e1[i0 + i]);
                            const float2 e2 = *reinterpret_cast<const float2*>(&fac.e2[i0 + i]);
                            const float2 o = fma2(e1, mul2(both2(f1), make_float2(x[i], x[i + 1])),
                                                  mul2(e2, mul2(both2(f2), make_float2(y[i], y[i + 1]))));
                            x[i] = o.x;
                            x[i + 1] = o.y;
                        }
                        if constexpr (OUT32) {
                            float* p = static_cast<float*>(a.out) + o0 + c + i0 * row_stride;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i0 + i < n) p[i * row_stride] = x[i];
                        } else {
                            // neighbouring lanes trade a value: even ones write two columns of row i, odd ones of row i + 1
                            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out) + o0 + (c & ~1) + (i0 + (c & 1)) * row_stride;
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float y1 = __shfl_xor_sync(0xffffffffu, (c & 1) ? x[i] : x[i + 1], 1);
                                const __nv_bfloat162 o = (c & 1) ? __floats2bfloat162_rn(y1, x[i + 1]) : __floats2bfloat162_rn(x[i], y1);
                                if (i0 + i + (c & 1) < n) *reinterpret_cast<__nv_bfloat162*>(p + i * row_stride) = o;
                            }
                        }
                        __syncwarp();
                    }
                }
                q0 += chunks;
            }
        } else
            for (int turn = 0; units.next(sm, a, ws, turn, u);) ++turn;
    }
    if (wait.dead) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
    ptx::tc_fence_before();
    chain_sync();
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TM_COLS);
    }
}

template <int DK, int DV, bool OUT32>
__global__ void __launch_bounds__(CHAIN_THREADS, 1) gdn_chain_kernel(const GdnArgs a, const __grid_constant__ CUtensorMap vmap, const Work ws)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    extern __shared__ __align__(1024) unsigned char dyn[];
    OneUnit one;
    Unit& u = one.u;
    u.h = blockIdx.x % a.Hv;
    u.seq = ranked_seq(a.cu_seqlens, a.N, blockIdx.x / a.Hv, &reinterpret_cast<ChainSmem<DK, DV>*>(dyn)->found);
    if (!gdn_unit(a, u.seq, u.begin, u.end, u.slot)) return;
    __shared__ uint32_t tmem;
    if (threadIdx.x / 32 == 8) ptx::tmem_alloc(&tmem, TM_COLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    run_chains<DK, DV, OUT32>(dyn, a, vmap, ws, tmem, one);
}

// ------------------------------------------------------------ chains beside prep
//
// A few long chains leave most SMs idle, and would start only when all of prep
// is done: one cooperative grid of a CTA an SM instead.  The first K CTAs start
// with the longest chains, the others with prep, three teams of warps each, in the order in which
// the chains come to need the slots; and whoever is done takes the next chain, longest
// first.  Prep waits for nobody, so the chains' waits for its slots end.
//
// K: as many chains as are longer than the work of all chains spread over all SMs.
// Those have to start before prep ends; were it fewer, one of them would end last
// alone, were it more, prep would be slower for nothing.  At most half of the CTAs.
constexpr int MERGED = 64;                    // sequences, two a lane
constexpr int BESIDE = PREP_CTAS * PREP;  // threads: as many teams of prep as CTAs of it fit on an SM
static_assert(BESIDE >= CHAIN_THREADS, "roles");

struct Plan {
    int order[MERGED];  // the sequences, longest first; those nothing is to be done for last
    int len[MERGED];    // chunks, by sequence
    int chains, first;  // K; sequences among the chains that start first
};

// One warp.
__device__ __forceinline__ void make_plan(Plan& p, const GdnArgs& a, int lane)
{
    int nc[2], total = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 32 * i;
        nc[i] = 0;
        if (s < a.N) {
            const int b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1], slot = a.slots ? a.slots[s] : s;
            if (b >= 0 && e > b && e <= a.T && slot >= 0 && slot < a.num_slots) nc[i] = (e - b + C - 1) / C;
        }
        p.len[s] = nc[i];
        total += nc[i];
    }
    total = __reduce_add_sync(0xffffffffu, total);
    __syncwarp();
    int r[2] = {0, 0}, above = 0;
    for (int k = 0; k < a.N; ++k) {
        const int l = p.len[k];
#pragma unroll
        for (int i = 0; i < 2; ++i) r[i] += l > nc[i] || (l == nc[i] && k < lane + 32 * i);
        above += (long long)l * gridDim.x > (long long)total * a.Hv;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < a.N) p.order[r[i]] = lane + 32 * i;
    if (lane == 0) {
        p.chains = (int)min((long long)above * a.Hv, (long long)gridDim.x / 2);
        p.first = (p.chains + a.Hv - 1) / a.Hv;
    }
}

// Prep's order: chunk 0 of the sequences whose chains start first, chunk 1 of
// those of them that have one, ..; then the other sequences, longest first, one after the other.
struct Order {
    int b[2], e[2], nc[2], seq[2];  // of the sequences at places lane and lane + 32 of the plan's order
    int first, most, total;         // of the ones that start first: how many, their most chunks, all their chunks
    int ends[2];                    // running sums of the others' chunks
    __device__ __forceinline__ int before(int c) const
    {
        return __reduce_add_sync(0xffffffffu, (lane() < first ? min(nc[0], c) : 0) + (lane() + 32 < first ? min(nc[1], c) : 0));
    }
    static __device__ __forceinline__ int lane() { return threadIdx.x & 31; }
    __device__ __forceinline__ Order(const Plan& p, const GdnArgs& a) : first(p.first), most(0)
    {
        int run[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = lane() + 32 * i;
            seq[i] = at < a.N ? p.order[at] : 0;
            nc[i] = at < a.N ? p.len[seq[i]] : 0;
            b[i] = a.cu_seqlens[seq[i]];
            e[i] = a.cu_seqlens[seq[i] + 1];
            if (at < first) most = max(most, nc[i]);
            run[i] = at < first ? 0 : nc[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, run[i], o);
                if (lane() >= o) run[i] += up;
            }
        }
        ends[0] = run[0];
        ends[1] = run[1] + __shfl_sync(0xffffffffu, run[0], 31);
        most = __reduce_max_sync(0xffffffffu, most);
        total = before(most);
    }
    // Task p: its slot and rows; false past the last.
    __device__ __forceinline__ bool task(int p, int& slot, int& r0, int& n) const
    {
        int at = -1, c;
        if (p < total) {
            int lo = 0, hi = most;  // before(lo) <= p < before(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (before(mid) <= p) lo = mid;
                else hi = mid;
            }
            c = lo;
            // longest first: the ones with more than c chunks are the first of the order
            at = p - before(lo);
        } else {
            p -= total;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t past = __ballot_sync(0xffffffffu, ends[i] > p);
                if (at < 0 && past) at = __ffs(past) - 1 + 32 * i;
            }
            if (at < 0) return false;
            const int l = at & 31, end = __shfl_sync(0xffffffffu, at < 32 ? ends[0] : ends[1], l);
            c = p - (end - __shfl_sync(0xffffffffu, at < 32 ? nc[0] : nc[1], l));
        }
        const int l = at & 31;
        const int bb = __shfl_sync(0xffffffffu, at < 32 ? b[0] : b[1], l), ee = __shfl_sync(0xffffffffu, at < 32 ? e[0] : e[1], l);
        slot = bb / C + __shfl_sync(0xffffffffu, at < 32 ? seq[0] : seq[1], l) + c;
        r0 = bb + c * C;
        n = min(C, ee - r0);
        return true;
    }
};

// Chain after chain, longest first: CTA i < K starts with chain i, the others are given out one by one.
struct TakenUnits {
    static constexpr bool BESIDE = true;
    const Plan* plan;
    template <class S> __device__ __forceinline__ bool next(S& sm, const GdnArgs& a, const Work& ws, int turn, Unit& out)
    {
        chain_sync();  // everyone is done with the unit before
        if (threadIdx.x == 0) {
            Unit& u = sm.unit;
            int i = turn == 0 && (int)blockIdx.x < plan->chains ? (int)blockIdx.x : -1;
            for (;; i = -1) {
                if (i < 0) i = plan->chains + atomicAdd(ws.taken, 1);
                if (i >= a.N * a.Hv) {
                    u.seq = -1;
                    break;
                }
                u.seq = plan->order[i / a.Hv];
                u.h = i % a.Hv;
                if (gdn_unit(a, u.seq, u.begin, u.end, u.slot)) break;
            }
        }
        chain_sync();
        out = sm.unit;
        return out.seq >= 0;
    }
};

template <int DK, int DV, bool OUT32, int HEADS>
__global__ void __launch_bounds__(BESIDE, 1)
gdn_beside_kernel(const GdnArgs a, const __grid_constant__ RowMaps maps, const Work ws)
{
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ Plan plan;
    __shared__ uint32_t tmem_at;
    // one allocation a CTA: 128 columns for a team of prep, then all of them for chains
    if (threadIdx.x < 32) make_plan(plan, a, threadIdx.x);
    else if (threadIdx.x / 32 == 8) ptx::tmem_alloc(&tmem_at, TM_COLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_at;
    if ((int)blockIdx.x >= plan.chains) {
        using S = PrepSmem<DK, HEADS>;
        constexpr int STRIDE = (sizeof(S) + 1023) / 1024 * 1024;
        const int team = threadIdx.x / PREP, t = threadIdx.x % PREP;
        S& sm = *reinterpret_cast<S*>(dyn + team * STRIDE);
        prep_setup(sm, t);
        team_sync(team);
        Waiter wait{false};
        const Order order(plan, a);
        const int groups = a.Hv / HEADS, teams = (gridDim.x - plan.chains) * PREP_CTAS;
        int turn = 0;
        for (long long i = (blockIdx.x - plan.chains) * PREP_CTAS + team;; i += teams, ++turn) {
            int slot, r0, n;
            if (!order.task((int)(i / groups), slot, r0, n)) break;
            const int h0 = (int)(i % groups) * HEADS;
            prep_task<DK, HEADS>(sm, a, maps, ws, slot, r0, n, h0, turn, team, tmem + team * 128, wait, t);
            if (t == 0) {
                ptx::bulk_wait_all();
                ptx::fence_proxy_async_global();
                __threadfence();
#pragma unroll
                for (int j = 0; j < HEADS; ++j) ptx::st_release_gpu(ws.ready + (long long)slot * a.Hv + h0 + j, 1);
            }
            team_sync(team);
        }
        if (wait.dead) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
        if (t == 0) {
            ptx::mbar_inval(&sm.loaded);
            ptx::mbar_inval(&sm.prod);
        }
        ptx::fence_proxy_async_smem();  // the chains' copies come into the same memory
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
    }
    if (threadIdx.x < CHAIN_THREADS) run_chains<DK, DV, OUT32>(dyn, a, maps.v, ws, tmem, TakenUnits{&plan});
    else set_regs<false, 24>();
}

// ------------------------------------------------------------ launch

// [T][width] bf16 rows with a row stride; boxes of 64 rows and `box` values.
bool encode_rows(CUtensorMap* m, const void* base, long long width, long long stride, int T, int box, bool swizzle)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)T};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {(cuuint32_t)box, C};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool OUT32>
cudaError_t launch_chain(const GdnArgs& a, const CUtensorMap& vmap, const Work& ws, cudaStream_t st)
{
    using S = ChainSmem<DK, DV>;
    constexpr int smem = sizeof(S);
    // operand tiles on the swizzle's 1024-byte period, barriers on 8
    static_assert(offsetof(S, work) % 1024 == 0 && offsetof(S, v) % 128 == 0 && offsetof(S, fac) % 16 == 0 && offsetof(S, loaded) % 8 == 0,
                  "alignment");
    static_assert(smem <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_chain_kernel<DK, DV, OUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(gdn_chain_kernel<DK, DV, OUT32>, a.N * a.Hv, CHAIN_THREADS, smem, st, a, vmap, ws);
}

template <int DK, int HEADS>
cudaError_t launch_prep(const GdnArgs& a, const RowMaps& maps, const Work& ws, long long slots, cudaStream_t st)
{
    using S = PrepSmem<DK, HEADS>;
    constexpr int smem = sizeof(S);
    static_assert(offsetof(S, t_hi) % 128 == 0 && offsetof(S, fac) % 16 == 0 && offsetof(S, m) % 16 == 0 &&
                  offsetof(S, xd) % 16 == 0 && offsetof(S, gates) % 16 == 0 &&
                  offsetof(S, col) % 16 == 0 && offsetof(S, loaded) % 8 == 0, "alignment");
    static_assert((smem + 1024) * PREP_CTAS <= 228 * 1024, "shared memory");
    static PerDeviceOnce once;
    const cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_prep_kernel<DK, HEADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(gdn_prep_kernel<DK, HEADS>, (unsigned)(slots * (a.Hv / HEADS)), PREP, smem, st, a, maps, ws);
}

template <int DK, int DV, bool OUT32, int HEADS>
cudaError_t launch_beside(const GdnArgs& a, const RowMaps& maps, const Work& ws, long long slots, cudaStream_t st)
{
    constexpr int prep = PREP_CTAS * (int)((sizeof(PrepSmem<DK, HEADS>) + 1023) / 1024 * 1024);
    constexpr int chain = (int)sizeof(ChainSmem<DK, DV>), smem = prep > chain ? prep : chain;
    static_assert(smem + sizeof(Plan) + 1024 <= 227 * 1024, "shared memory");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(gdn_beside_kernel<DK, DV, OUT32, HEADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    if ((e = cudaMemsetAsync(ws.ready, 0, (slots * a.Hv + 1) * sizeof(int), st)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = sm_count();
    cfg.blockDim = BESIDE;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_beside_kernel<DK, DV, OUT32, HEADS>, a, maps, ws);
}

template <int DK, int DV, bool OUT32>
cudaError_t launch_dv(const GdnArgs& a, const RowMaps& maps, const Work& ws, long long slots, cudaStream_t st)
{
    // Two heads a team (their rows, products and norms once): 32768 rows as eight prompts take
    // 725 us, 840 with one; one prompt 1350 and 1333.
    const bool pairs = a.Hv / a.Hk % 2 == 0, waves = slots * a.Hv > PREP_CTAS * sm_count();
    // Chains beside prep where prep is more than one wave of CTAs, in us (in brackets: one after the
    // other).  32768 rows of 32 heads: one prompt 1350 (1683); mixed lengths of 8 prompts 725 (881), 12 709 (789),
    // 16 707 (670), 32 741 (703), 64 803 (777); equal ones of 2 693 (1014), 4 912 (689), 8 734 (698), 16 744 (711),
    // 64 775 (762).  Of 4 heads: mixed lengths of 4 to 64 prompts 533 to 130 (555 to 158), equal ones of 16 128 (148),
    // 24 178 (124), 32 164 (109), 64 120 (119).  8192 rows of 12 heads: mixed lengths of 8 120 (126), 24 94 (97), 32 95
    // (89), 64 111 (106).  333 rows of 8 heads, not a wave: 42 (24).  So it gains where some chains are longer than the
    // others or there are few of them, up to a third, and loses some 5 % where there are several equal ones for every
    // SM and up to a third where there is about one: the lengths are on the device, where this choice cannot see them.
    // That grid's chains wait for prep on other SMs, so all of its CTAs have to be resident: on a stream of a
    // partition of the device one after the other, with the same bits.
    if (a.N <= MERGED && waves && stream_sm_count(st) >= sm_count())
        return pairs ? launch_beside<DK, DV, OUT32, 2>(a, maps, ws, slots, st) : launch_beside<DK, DV, OUT32, 1>(a, maps, ws, slots, st);
    // (in one wave all single heads run at once)
    const cudaError_t e = pairs && waves ? launch_prep<DK, 2>(a, maps, ws, slots, st) : launch_prep<DK, 1>(a, maps, ws, slots, st);
    return e != cudaSuccess ? e : launch_chain<DK, DV, OUT32>(a, maps.v, ws, st);
}

template <int DK, bool OUT32> cudaError_t launch(const GdnArgs& a, int dv, cudaStream_t st)
{
    using L = Slot<DK>;
    RowMaps maps;
    if (!encode_rows(&maps.q, a.q, (long long)a.Hk * DK, a.qs, a.T, 64, true) ||
        !encode_rows(&maps.k, a.k, (long long)a.Hk * DK, a.ks, a.T, 64, true) ||
        !encode_rows(&maps.v, a.v, (long long)a.Hv * dv, a.vs, a.T, dv, false))
        return cudaErrorInvalidValue;
    const long long slots = slot_count(a.N, a.T);
    Work ws;
    ws.kq = static_cast<unsigned char*>(a.workspace);
    ws.v = ws.kq + slots * a.Hk * L::KQ;
    ws.ready = reinterpret_cast<int*>(ws.v + slots * a.Hv * L::V);
    ws.taken = ws.ready + slots * a.Hv;
    if (dv == 128) return launch_dv<DK, 128, OUT32>(a, maps, ws, slots, st);
    if (dv == 64) return launch_dv<DK, 64, OUT32>(a, maps, ws, slots, st);
    return launch_dv<DK, 32, OUT32>(a, maps, ws, slots, st);
}

}  // namespace
}  // namespace kda
