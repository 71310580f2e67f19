// kda_paged_token.cu -- attention of single bf16 rows over a paged cache.
//
// Every cached value is read once for the G query heads that share it, so HBM bandwidth is the bound: a row's
// products are a handful a byte.  All that matters is that every SM keeps loading until the last byte: the tiles
// of all (sequence, key head) pairs form one line, and each of CTAS CTAs takes an equal stretch of it, whatever the
// lengths.  A pair within one stretch is written out; one that stretches cut leaves a part in the workspace for each
// of them, and token_join_kernel adds the parts.
// A warp loads (tensor copies, a ring of tiles); teams of warps that take the tiles in turn hold 16 tokens of a tile
// a warp: scores and values by mma.sync with up to 16 heads as rows (a tcgen05 tile would have 128 of them, nearly all empty), weights
// in two bf16 parts (2^-17 of each: the outputs keep fp32's places), running maximum and sum of each warp by itself, joined at the pair's end.
// Measured: 64 sequences of up to 32768 tokens, eight key heads of 128 (4.3 GB), 627 us, 6.9 TB/s; 128 of 2048 tokens, two key heads of
// 256 in pages of 16 (0.54 GB), 93 us, 5.8 TB/s with the start and the join (10 us together); fp32, 64 of 4096 tokens, 341 us, 6.3 TB/s.  One sequence of
// 32768 tokens (134 MB) takes 30 us, of which the join is 6; 250 sequences of 1 to 100 tokens 45.
#include <cuda.h>

#include "kda_paged.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int CTAS = 152;     // one an SM
constexpr int KNOWN = 512;    // sequences whose lengths a CTA keeps
constexpr float LAG = 8.f;

// What the stretches leave for token_join_kernel.
struct Cut {
    long long line;            // tiles in all
    int seq, unit, last;       // the unit that begins in this stretch and ends in that of CTA `last`; seq < 0: none
    int pad;
};
struct TokenWork {
    Cut* cut;                  // [CTAS]
    float2* ml;                // [CTAS][2][rows]: largest score (in powers of two) and sum of the weights;
    float* o;                  // [CTAS][2][rows][D]   0: of a unit that began before, 1: of the one that goes on
};

// Places for a unit's heads: eight (a column block of a product) or sixteen; a group has no more (paged_token_wanted).
int unit_rows(const PagedArgs& a) { return a.G <= 8 ? 8 : 16; }

size_t lay_out(TokenWork& w, const PagedArgs& a)
{
    const size_t rows = unit_rows(a);
    unsigned char* p = static_cast<unsigned char*>(a.workspace);
    size_t at = 0;
    const auto take = [&](size_t n) {
        unsigned char* x = p ? p + at : nullptr;
        at += (n + 255) / 256 * 256;
        return x;
    };
    w.cut = reinterpret_cast<Cut*>(take(sizeof(Cut) * CTAS));
    w.ml = reinterpret_cast<float2*>(take(sizeof(float2) * CTAS * 2 * rows));
    w.o = reinterpret_cast<float*>(take(sizeof(float) * CTAS * 2 * rows * (size_t)a.D));
    return at;
}

// Teams of TEAM warps, 16 tokens of a tile each, take the tiles in turn.  A stage of the ring belongs to one team (their
// number divides the stages'), so that whoever waits for a stage has waited for each of its uses: parities tell two apart, not three.
template <typename IO, int D, int HB> struct Token {
    static constexpr int SIZE = sizeof(IO), WIDE = 128 / SIZE;   // values of 128 bytes
    static constexpr int DP = D < WIDE ? WIDE : D, BLOCKS = DP / WIDE;
    static constexpr int ROWS = 8 * HB;
    static constexpr int TEAM = D * SIZE == 1024 ? 1 : D * SIZE == 512 ? 2 : 4;
    static constexpr int WARPS = TEAM == 1 ? 6 : HB == 1 ? 12 : TEAM == 2 ? 6 : 8, TEAMS = WARPS / TEAM;  // as registers allow
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int KEYS = 16 * TEAM;                         // tokens of a tile
    static constexpr int HALF = KEYS * DP * SIZE, STAGE = 2 * HALF;  // keys, then values
    static constexpr int STAGES = STAGE <= 16384 ? 12 : 6;
    static constexpr int CH = D == 128 && HB == 1 && SIZE == 2 ? 64 : WARPS * 2 < ROWS ? 16 : 32;  // as shared memory and threads allow
    static constexpr int QS = D * SIZE + 16;                       // bytes of a row of q: eight rows in distinct banks
    static_assert(STAGES % TEAMS == 0, "a stage belongs to one team");
    static_assert(WARPS * 32 >= ROWS * CH / 2, "two channels a thread");
    struct Smem {
        unsigned char ring[STAGES * STAGE];
        unsigned char q[2][ROWS * QS];
        float o[WARPS][ROWS * (CH + 4)];  // CH channels of every warp's sums at a time
        float2 ml[WARPS][ROWS];
        float w[SIZE == 4 ? WARPS : 1][16 * 8];  // fp32 rows: weights of 16 tokens and eight heads
        uint64_t full[STAGES], empty[STAGES], qfull[2], qempty[2];
        int kv[KNOWN];                    // lengths from the stretch's first sequence on, -1: skipped
        long long sum[WARPS + 1];
        uint32_t hidden[STAGES];
        int first, dead;
        long long offset;
    };
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// An 8 x 8 block of 16-bit values, turned.
__device__ __forceinline__ uint32_t turn8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int x, int y, int z, int w, int v, uint64_t* bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(
            ptx::smem_u32(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(ptx::smem_u32(bar)), "l"(policy)
        : "memory");
}

// Tokens lo .. kv - 1 are seen; tiles count from lo's page (or tile within a page) on.
template <int KEYS> struct Span {
    int lo, start, n;
    __device__ __forceinline__ Span(const PagedArgs& a, int kv)
    {
        lo = a.window && kv > a.window ? kv - a.window : 0;
        start = lo & ~(min(KEYS, 1 << a.page_shift) - 1);
        n = kv < 0 ? 0 : max(1, (kv - start + KEYS - 1) / KEYS);
    }
};

__device__ __forceinline__ int length_of(const PagedArgs& a, int s, int* fault)
{
    int begin, end, kv;
    return paged_seq(a, s, begin, end, kv, fault) ? kv : -1;
}

__device__ __forceinline__ long long stretch(long long line, int c) { return line * c / CTAS; }
__device__ __forceinline__ int owner(long long line, long long x) { return (int)(((x + 1) * CTAS + line - 1) / line) - 1; }

// A CTA's walk along its stretch, unit after unit.
struct Walk {
    int s, kv, u;            // sequence, its tokens, key head
    int lo, start, n;        // as in Span
    int t0, t1;              // tiles of the unit in this stretch
    long long left;          // tiles of the stretch from t0 on
};

template <int KEYS, class S> __device__ __forceinline__ void enter(const PagedArgs& a, const S& sm, Walk& w)
{
    while (true) {  // sequences without tokens are passed over; one with tokens follows while tiles are left
        const int i = w.s - sm.first;
        int f = 0;
        if (w.s >= a.N) {  // lengths that changed under the call
            w.left = w.kv = 0;
            break;
        }
        w.kv = i < KNOWN ? sm.kv[i] : length_of(a, w.s, &f);
        if (w.kv >= 0) break;
        ++w.s;
    }
    const Span<KEYS> x(a, w.kv);
    w.lo = x.lo;
    w.start = x.start;
    w.n = x.n;
}
template <int KEYS, class S> __device__ __forceinline__ void begin_walk(const PagedArgs& a, const S& sm, Walk& w, long long tiles)
{
    w.s = sm.first;
    w.left = tiles;
    if (tiles <= 0) return;
    enter<KEYS>(a, sm, w);
    w.u = (int)(sm.offset / w.n);
    w.t0 = (int)(sm.offset % w.n);
    w.t1 = (int)min((long long)w.n, w.t0 + w.left);
}
template <int KEYS, class S> __device__ __forceinline__ void next_unit(const PagedArgs& a, const S& sm, Walk& w)
{
    w.left -= w.t1 - w.t0;
    if (w.left <= 0) return;
    if (++w.u == a.Hkv) {
        w.u = 0;
        ++w.s;
        enter<KEYS>(a, sm, w);
    }
    w.t0 = 0;
    w.t1 = (int)min((long long)w.n, w.left);
}

template <typename IO, int D, int HB> __global__ void __launch_bounds__(Token<IO, D, HB>::THREADS, 1)
paged_token_kernel(const PagedArgs a, const TokenWork work, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using L = Token<IO, D, HB>;
    constexpr bool F32 = sizeof(IO) == 4;
    constexpr int ROWS = L::ROWS, STAGES = L::STAGES, BLOCKS = L::BLOCKS, KEYS = L::KEYS, WARPS = L::WARPS, TEAM = L::TEAM, TT = L::THREADS;
    extern __shared__ __align__(1024) unsigned char raw[];
    auto& s = *reinterpret_cast<typename L::Smem*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(&s.full[i], 1);
            ptx::mbar_init(&s.empty[i], TEAM);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s.qfull[i], 1);
            ptx::mbar_init(&s.qempty[i], WARPS);
        }
        s.dead = 0;
        ptx::fence_mbar_init();
    }
    for (int i = tid; i < (int)sizeof(s.q) / 16; i += TT) reinterpret_cast<uint4*>(s.q)[i] = make_uint4(0, 0, 0, 0);  // rows without a head stay zero
    if (tid == 32) {  // the maps are the launch's own arguments: no need to wait for them
        ptx::prefetch_map(&kmap);
        ptx::prefetch_map(&vmap);
    }
    ptx::fence_proxy_async_smem();
    ptx::grid_dependency_wait();

    // ---- the stretch: tiles before each thread's run of sequences, then the sequence in which the stretch begins
    const int per = (a.N + TT - 1) / TT, s0 = min(tid * per, a.N), s1 = min(s0 + per, a.N);
    long long mine = 0;
    int fault = 0;
    int known = -1;
    for (int i = s0; i < s1; ++i) {
        known = length_of(a, i, &fault);
        mine += Span<KEYS>(a, known).n;
    }
    if (blockIdx.x == 0 && fault) flag_status(a.dev_status, fault);
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) s.sum[warp] = before;
    if (tid == 0) s.first = a.N;
    __syncthreads();
    long long line = 0;
    for (int w = 0; w < TT / 32; ++w) {
        if (w < warp) before += s.sum[w];
        line += s.sum[w];
    }
    before -= mine;
    line *= a.Hkv;
    before *= a.Hkv;
    const long long x0 = stretch(line, blockIdx.x), x1 = stretch(line, blockIdx.x + 1);
    if (x0 < x1 && before <= x0 && x0 < before + mine * a.Hkv) {
        int i = s0, f = 0;
        for (;; ++i) {
            const int n = Span<KEYS>(a, length_of(a, i, &f)).n;
            if (x0 < before + (long long)n * a.Hkv) break;
            before += (long long)n * a.Hkv;
        }
        s.first = i;
        s.offset = x0 - before;
    }
    __syncthreads();
    for (int i = tid; i < KNOWN; i += TT) {
        int f = 0;
        if (per > 1 || s.first + i >= a.N) s.kv[i] = s.first + i < a.N ? length_of(a, s.first + i, &f) : -1;
    }
    if (per == 1 && tid < a.N && tid >= s.first && tid - s.first < KNOWN) s.kv[tid - s.first] = known;  // a sequence a thread: it is at hand
    __syncthreads();
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ptx::mbar_wait(bar, parity & 1, a.polls) && !*reinterpret_cast<volatile int*>(&s.dead)) return true;
        *reinterpret_cast<volatile int*>(&s.dead) = 1;
        return false;
    };
    Walk w;
    begin_walk<KEYS>(a, s, w, x1 - x0);
    bool ok = true;
    if (warp == WARPS) {
        // ---- loads
        ok = (int)blockIdx.x != a.stalled;
        const uint64_t once = ptx::policy_evict_first();
        const int box = min(KEYS, 1 << a.page_shift), boxes = KEYS / box;
        uint32_t use = 0, unit = 0;
        for (; w.left > 0 && ok; next_unit<KEYS>(a, s, w), ++unit) {
            const int h = w.u;
            if (!(ok = wait(&s.qempty[unit & 1], (unit >> 1) + 1))) break;
            if (lane == 0) ptx::mbar_arrive_expect_tx(&s.qfull[unit & 1], a.G * D * L::SIZE);
            __syncwarp();
            if (lane < a.G)
                ptx::bulk_g2s(s.q[unit & 1] + lane * L::QS, static_cast<const IO*>(a.q) + w.s * a.q_stride + (long long)(h * a.G + lane) * D,
                              D * L::SIZE, &s.qfull[unit & 1]);
            for (int t = w.t0; t < w.t1; ++t, ++use) {
                const int stage = use % STAGES, k0 = w.start + t * KEYS, tok = k0 + lane % boxes * box;
                const bool in = tok < w.kv;
                int page = 0;
                if (in) page = a.pages[(long long)w.s * a.width + (tok >> a.page_shift)];
                const bool gone = in && (page < 0 || page >= a.num_pages);
                const uint32_t hide = __ballot_sync(0xffffffffu, gone && lane < boxes);
                const int n = __popc(__ballot_sync(0xffffffffu, in && lane < boxes));
                if (!(ok = wait(&s.empty[stage], use / STAGES + 1))) break;
                if (lane == 0) {
                    s.hidden[stage] = hide;
                    if (hide) flag_status(a.dev_status, KDA_DEV_BAD_PAGE);
                    ptx::mbar_arrive_expect_tx(&s.full[stage], n * box * 128 * BLOCKS * 2);
                }
                __syncwarp();
                // a copy a page of keys and of values; each lane holds the page of box lane % boxes
                if (lane < 2 * boxes && in)
                    tma_load_5d(s.ring + stage * L::STAGE + lane / boxes * L::HALF + lane % boxes * box * (L::DP * L::SIZE), lane < boxes ? &kmap : &vmap, 0,
                                tok & ((1 << a.page_shift) - 1), 0, h, gone ? -1 : page, &s.full[stage], once);
            }
        }
        if (!ok && lane == 0) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
        // what is on its way has to land first (it has, unless those who wait for it gave up)
        for (uint32_t u = use > STAGES ? use - STAGES : 0; u < use; ++u) ptx::mbar_wait(&s.full[u % STAGES], (u / STAGES) & 1, PAGED_POLLS);
        for (uint32_t u = unit > 2 ? unit - 2 : 0; u < unit; ++u) ptx::mbar_wait(&s.qfull[u & 1], (u >> 1) & 1, PAGED_POLLS);
    } else {
        const int team = warp / TEAM, k16 = warp % TEAM * 16;  // this warp's tokens of a tile
        const float c = a.scale * 1.4426950408889634f;
        uint32_t use = 0, unit = 0;
        const uint32_t ring = ptx::smem_u32(s.ring);
        if (tid == 0) work.cut[blockIdx.x].seq = -1;
        // (a wait that ran out: the warps go on without waiting and without tiles, so that they still meet at the barriers; a unit that a warp gave up on
        // is written nowhere, PART_LOST in its place)
        for (; w.left > 0; next_unit<KEYS>(a, s, w), ++unit) {
            const int h = w.u, rows = a.G;
            ok = ok && wait(&s.qfull[unit & 1], unit >> 1);
            // tokens are the products' rows, heads their columns: S^T = K Q^T, O^T += V^T W^T
            const uint32_t qbase = ptx::smem_u32(s.q[unit & 1]) + (lane & 7) * L::QS + (lane >> 3) * 16;
            constexpr bool KEEP = !F32 && D * HB <= 128;  // more than that comes from shared memory each time: registers
            uint32_t qf[HB][KEEP ? D / 32 : 1][4];
            if constexpr (KEEP) {
#pragma unroll
                for (int b = 0; b < HB; ++b)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) ldsm(qf[b][k], qbase + b * 8 * L::QS + k * 64);
            }
            float o[F32 ? 1 : HB][F32 ? 1 : D / 16][4], m[HB][2], l[HB][2];  // of this lane's two heads (a block)
            // fp32 rows: all eight heads, D / 32 channels a lane
            constexpr int PER = D / 32;
            float of[F32 ? 8 : 1][F32 ? PER : 1], mf[F32 ? 8 : 1], lf[F32 ? 8 : 1];
            if constexpr (F32) {
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    mf[g] = -INFINITY;
                    lf[g] = 0.f;
#pragma unroll
                    for (int i = 0; i < PER; ++i) of[g][i] = 0.f;
                }
            }
#pragma unroll
            for (int b = 0; b < HB; ++b) {
                m[b][0] = m[b][1] = -INFINITY;
                l[b][0] = l[b][1] = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if constexpr (!F32) o[b][i][e] = 0.f;
            }
            for (int t = w.t0; t < w.t1; ++t, ++use) {
                if (use % L::TEAMS != (uint32_t)team) continue;
                const int stage = use % STAGES, k0 = w.start + t * KEYS + k16;
                if (!ok || !(ok = wait(&s.full[stage], use / STAGES))) continue;
                const uint32_t hide = *reinterpret_cast<volatile uint32_t*>(&s.hidden[stage]);
                // a box holds its tokens' first 64 channels, then the next 64 ...
                const int box_shift = min(a.page_shift, KEYS == 64 ? 6 : KEYS == 32 ? 5 : 4), blk_bytes = 128 << box_shift;
                const uint32_t kb = ring + stage * L::STAGE + (k16 >> box_shift) * (blk_bytes * BLOCKS) + (k16 & ((1 << box_shift) - 1)) * 128, vb = kb + L::HALF;
                const bool gone = (hide >> (k16 >> box_shift)) & 1;
                const bool part = k0 + 16 > w.kv || k0 < w.lo || gone;
                if (part) {
                    // values of places that the row does not see, whatever lies there: zeros
                    unsigned char* v = s.ring + (vb - ring);
                    for (int i = lane; i < 16 * 8 * BLOCKS; i += 32) {
                        const int r = i / 8 % 16, blk = i / 128;
                        if (k0 + r >= w.kv || k0 + r < w.lo || gone) *reinterpret_cast<uint4*>(v + blk * blk_bytes + r * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                if constexpr (F32) {
                    // scores: two lanes a token, half of every 32 channels each
                    const int tk = lane >> 1, half = lane & 1, tok = k0 + tk;
                    const unsigned char* kr = s.ring + (kb - ring) + tk * 128;
                    const unsigned char* qr = s.q[unit & 1];
                    float sc[8] = {};
#pragma unroll 4
                    for (int i = 0; i < D / 8; ++i) {
                        const int ch = half * 4 + i % 4, blk = i / 4;
                        const float4 k = *reinterpret_cast<const float4*>(kr + blk * blk_bytes + ((ch ^ (tk & 7)) << 4));
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (g < rows) {
                                const float4 q = *reinterpret_cast<const float4*>(qr + g * L::QS + blk * 128 + ch * 16);
                                sc[g] = fmaf(q.w, k.w, fmaf(q.z, k.z, fmaf(q.y, k.y, fmaf(q.x, k.x, sc[g]))));
                            }
                    }
                    const bool seen = !(part && (gone || tok >= w.kv || tok < w.lo));
                    bool grow = false;
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        if (g < rows) {
                            sc[g] += __shfl_xor_sync(0xffffffffu, sc[g], 1);
                            sc[g] = seen ? c * sc[g] : -INFINITY;
                            grow |= sc[g] > mf[g] + LAG;
                        }
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (g < rows) {
                                float x = sc[g];
#pragma unroll
                                for (int d = 2; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                                const float next = fmaxf(mf[g], x), f = next == -INFINITY ? 1.f : exp2_sfu(mf[g] - next);
                                mf[g] = next;
                                lf[g] *= f;
#pragma unroll
                                for (int i = 0; i < PER; ++i) of[g][i] *= f;
                            }
                    }
                    float* wr = s.w[warp];
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        if (g < rows) {
                            const float x = exp2_sfu(sc[g] - (mf[g] == -INFINITY ? 0.f : mf[g]));
                            if (half == 0) {
                                lf[g] += x;
                                wr[tk * 8 + g] = x;
                            }
                        }
                    __syncwarp();
                    const unsigned char* vr = s.ring + (vb - ring);
#pragma unroll 4
                    for (int t16 = 0; t16 < 16; ++t16) {
                        float v[PER];
                        if constexpr (PER >= 4) {
#pragma unroll
                            for (int i = 0; i < PER; i += 4)
                                *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(vr + (i + lane / 8) * blk_bytes + t16 * 128 + ((lane % 8 ^ (t16 & 7)) << 4));
                        } else {
                            const int at = lane * PER;
#pragma unroll
                            for (int i = 0; i < PER; ++i)
                                v[i] = *reinterpret_cast<const float*>(vr + at / 32 * blk_bytes + t16 * 128 + ((at % 32 / 4 ^ (t16 & 7)) << 4) + (at % 4 + i) * 4);
                        }
                        const float4 w0 = *reinterpret_cast<const float4*>(wr + t16 * 8), w1 = *reinterpret_cast<const float4*>(wr + t16 * 8 + 4);
                        const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (g < rows)
#pragma unroll
                                for (int i = 0; i < PER; ++i) of[g][i] = fmaf(ww[g], v[i], of[g][i]);
                    }
                } else {
                float sc[2][HB][4] = {};  // even and odd steps apart: half the latency
                {
                    const int r = lane & 15, ch = lane >> 4;
                    const uint32_t row = kb + r * 128;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t x[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) ldsm(x[i], row + (k / 2) * blk_bytes + (((k % 2 * 4 + i * 2 + ch) ^ (r & 7)) << 4));
#pragma unroll
                        for (int b = 0; b < HB; ++b) {
                            uint32_t q[4];
                            if constexpr (!KEEP) ldsm(q, qbase + b * 8 * L::QS + k * 64);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if constexpr (KEEP) mma16816(sc[i][b], x[i], qf[b][k][2 * i], qf[b][k][2 * i + 1]);
                                else mma16816(sc[i][b], x[i], q[2 * i], q[2 * i + 1]);
                            }
                        }
                    }
                }
                bool grow = false;
                float top[HB][2];
#pragma unroll
                for (int b = 0; b < HB; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[0][b][e] += sc[1][b][e];
                        const int tok = k0 + lane / 4 + (e & 2) * 4;
                        if (part && (gone || tok >= w.kv || tok < w.lo)) sc[0][b][e] = -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[b][e] = c * fmaxf(sc[0][b][e], sc[0][b][e + 2]);
                        grow |= top[b][e] > m[b][e] + LAG;
                    }
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int b = 0; b < HB; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = top[b][e];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                            const float next = fmaxf(m[b][e], x), f = next == -INFINITY ? 1.f : exp2_sfu(m[b][e] - next);
                            m[b][e] = next;
                            l[b][e] *= f;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                o[b][j][e] *= f;
                                o[b][j][e + 2] *= f;
                            }
                        }
                }
                uint32_t hi[HB][2], lo[HB][2];
#pragma unroll
                for (int b = 0; b < HB; ++b) {
                    const float base0 = m[b][0] == -INFINITY ? 0.f : m[b][0], base1 = m[b][1] == -INFINITY ? 0.f : m[b][1];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // tokens lane / 4, and eight on
                        const float x = exp2_sfu(fmaf(sc[0][b][2 * i], c, -base0)), y = exp2_sfu(fmaf(sc[0][b][2 * i + 1], c, -base1));
                        l[b][0] += x;
                        l[b][1] += y;
                        const uint32_t p = pack_bf16(x, y);
                        hi[b][i] = turn8(p);
                        lo[b][i] = turn8(pack_bf16(x - __uint_as_float(p << 16), y - __uint_as_float(p & 0xffff0000u)));
                    }
                }
                {
                    const int r = (lane & 7) + (lane >> 4) * 8, ch = (lane >> 3) & 1;
                    const uint32_t row = vb + r * 128;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t x[4];
                        ldsm_t(x, row + (j / 4) * blk_bytes + ((((j % 4) * 2 + ch) ^ (r & 7)) << 4));
#pragma unroll
                        for (int b = 0; b < HB; ++b) mma16816(o[b][j], x, hi[b][0], hi[b][1]);
#pragma unroll
                        for (int b = 0; b < HB; ++b) mma16816(o[b][j], x, lo[b][0], lo[b][1]);
                    }
                }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s.empty[stage]);
            }
            // ---- the warps' sums together
            if constexpr (F32) {
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    lf[g] = warp_sum(lf[g]);
                    if (lane == 0) s.ml[warp][g] = make_float2(mf[g], ok ? lf[g] : PART_LOST);
                }
            } else {
#pragma unroll
            for (int b = 0; b < HB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
                    if (lane < 4) s.ml[warp][b * 8 + lane * 2 + e] = make_float2(m[b][e], ok ? l[b][e] : PART_LOST);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.qempty[unit & 1]);
            asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
            float ff[F32 ? 8 : 1];
            if constexpr (F32) {
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    float top = -INFINITY;
                    for (int x = 0; x < WARPS; ++x) top = fmaxf(top, s.ml[x][g].x);
                    ff[g] = mf[g] == -INFINITY ? 0.f : exp2_sfu(mf[g] - top);
                }
            }
            float f[HB][2];
#pragma unroll
            for (int b = 0; b < HB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = -INFINITY;
                    for (int x = 0; x < WARPS; ++x) top = fmaxf(top, s.ml[x][b * 8 + (lane & 3) * 2 + e].x);
                    f[b][e] = m[b][e] == -INFINITY ? 0.f : exp2_sfu(m[b][e] - top);
                }
            // two of CH channels of a row at a time, by a thread each
            constexpr int CH = L::CH;
            const int row = tid / (CH / 2), ch = tid % (CH / 2) * 2;  // (threads past the last row have none)
            float top = -INFINITY, sum = 0.f;
            bool lost = false;
            for (int x = 0; x < WARPS; ++x) {
                top = fmaxf(top, s.ml[x][row % ROWS].x);
                lost |= s.ml[x][row % ROWS].y < 0.f;
            }
            const bool in = row < rows && !lost;
            const float base = top == -INFINITY ? 0.f : top;  // (warps that met only NaN have no maximum, but their sum)
            for (int x = 0; x < WARPS; ++x) sum += s.ml[x][row % ROWS].y * exp2_sfu(s.ml[x][row % ROWS].x - base);
            const bool whole = w.t0 == 0 && w.t1 == w.n;
            const int slot = w.t0 == 0 ? 1 : 0;
            const size_t head = (size_t)w.s * a.Hq + h * a.G + row, cell = ((size_t)blockIdx.x * 2 + slot) * ROWS + row;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < D; e += CH) {
                if constexpr (F32) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int at = PER >= 4 ? i / 4 * 128 + lane * 4 + i % 4 : lane * PER + i;
                        if (at / CH == e / CH)
#pragma unroll
                            for (int g = 0; g < 8; ++g) s.o[warp][g * (CH + 4) + at % CH] = of[g][i] * ff[g];
                    }
                } else {
#pragma unroll
                for (int b = 0; b < HB; ++b)
#pragma unroll
                    for (int j = 0; j < CH / 16; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s.o[warp][(b * 8 + (lane & 3) * 2 + (i & 1)) * (CH + 4) + j * 16 + lane / 4 + (i & 2) * 4] = o[b][e / 16 + j][i] * f[b][i & 1];
                }
                asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
                float2 y = make_float2(0.f, 0.f);
                if (row < ROWS)
#pragma unroll
                    for (int x = 0; x < WARPS; ++x) y = add2(y, *reinterpret_cast<const float2*>(&s.o[x][row * (CH + 4) + ch]));
                if (in) {
                    if (whole && F32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + head * D + e + ch) =
                        sum == 0.f ? make_float2(0.f, 0.f) : make_float2(y.x * inv, y.y * inv);
                    else if (whole) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + head * D + e + ch) =
                        sum == 0.f ? 0u : pack_bf16(y.x * inv, y.y * inv);
                    else *reinterpret_cast<float2*>(work.o + cell * D + e + ch) = y;
                }
                asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
            }
            if (row < rows && ch == 0) {
                if (!whole) work.ml[cell] = make_float2(top, lost ? PART_LOST : sum);
                else if (a.lse && in) a.lse[head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
            }
            if (w.t0 == 0 && !whole && tid == 0) {
                const long long last = x1 - 1 + (w.n - w.t1);  // the unit's last tile in the line
                work.cut[blockIdx.x] = {line, w.s, w.u, owner(line, last), 0};
            }
        }
        if (!ok && lane == 0) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
    }
    __syncthreads();
}

// A warp joins the parts of one row: part s has its maximum and sum at ml(s) and its D values at o(s), both
// null for a part without any.  Returns the maximum and the sum (PART_LOST where a part is), and in y the lane's D / 32 neighbouring values, not divided.
template <int D, class ML, class O> __device__ __forceinline__ float2 join_row(int parts, ML&& ml, O&& o, float (&y)[D / 32])
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f;
    bool lost = false;
    for (int s = lane; s < parts; s += 32)
        if (const float2* x = ml(s)) {
            m = fmaxf(m, x->x);
            lost |= x->y < 0.f;
        }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int e = 0; e < PER; ++e) y[e] = 0.f;
    for (int s0 = 0; s0 < parts; s0 += 32) {
        float f = 0.f;
        const float2* x = s0 + lane < parts ? ml(s0 + lane) : nullptr;
        if (x) {
            f = exp2f(x->x - base);
            l += f * x->y;
        }
        const int n = min(32, parts - s0);
#pragma unroll 8
        for (int s = 0; s < n; ++s) {
            const float g = __shfl_sync(0xffffffffu, f, s);
            const float* v = o(s0 + s);
            if (!v) continue;
            if constexpr (PER >= 4) {
#pragma unroll
                for (int e = 0; e < PER; e += 4) {
                    const float4 z = *reinterpret_cast<const float4*>(v + lane * PER + e);
                    y[e] = fmaf(g, z.x, y[e]);
                    y[e + 1] = fmaf(g, z.y, y[e + 1]);
                    y[e + 2] = fmaf(g, z.z, y[e + 2]);
                    y[e + 3] = fmaf(g, z.w, y[e + 3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) y[e] = fmaf(g, v[lane * PER + e], y[e]);
            }
        }
    }
    l = warp_sum(l);
    return make_float2(m, __any_sync(0xffffffffu, lost) ? PART_LOST : l);
}
// The joined row to out and lse (row: of [T][Hq]).
template <typename IO, int D> __device__ __forceinline__ void write_row(const PagedArgs& a, size_t row, float2 ml, const float (&y)[D / 32])
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    if (ml.y < 0.f) return;
    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
    IO* out = static_cast<IO*>(a.out) + row * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) stv(out + e, ml.y == 0.f ? 0.f : y[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.69314718055994531f;
}

// The parts of the unit that begins in stretch blockIdx.x and goes on: a warp a row.
template <typename IO, int D, int ROWS> __global__ void __launch_bounds__(32 * ROWS) token_join_kernel(const PagedArgs a, const TokenWork work)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const Cut cut = work.cut[blockIdx.x];
    if (cut.seq < 0) return;
    const int row = threadIdx.x >> 5;
    // stretches without a tile (fewer tiles than stretches) left nothing
    const auto used = [&](int s) { return stretch(cut.line, blockIdx.x + s) < stretch(cut.line, blockIdx.x + s + 1); };
    const auto cell = [&](int s) { return ((size_t)(blockIdx.x + s) * 2 + (s == 0)) * ROWS + row; };
    float y[D / 32];
    const float2 ml = join_row<D>(cut.last - (int)blockIdx.x + 1, [&](int s) { return used(s) ? work.ml + cell(s) : nullptr; },
                                         [&](int s) { return used(s) ? work.o + cell(s) * D : nullptr; }, y);
    write_row<IO, D>(a, (size_t)cut.seq * a.Hq + cut.unit * a.G + row, ml, y);
}

// [num_pages][Hkv][D / 64][page_size][64] (fp32: 32 values, 128 bytes either way) by the cache's strides; boxes of a page's (or a tile's) tokens and all channels of one head.
bool encode_cache(CUtensorMap* m, const void* base, const PagedArgs& a, int keys, int size)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t P = (cuuint64_t)1 << a.page_shift, wide = 128 / size, blocks = std::max<cuuint64_t>(1, a.D / wide);
    const cuuint64_t dims[5] = {std::min<cuuint64_t>(a.D, wide), P, blocks, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)a.token_stride * size, 128, (cuuint64_t)a.head_stride * size, (cuuint64_t)a.page_stride * size};
    const cuuint32_t box[5] = {(cuuint32_t)wide, (cuuint32_t)std::min<cuuint64_t>(P, keys), (cuuint32_t)blocks, 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename IO, int D, int HB> cudaError_t launch(const PagedArgs& a, cudaStream_t st)
{
    using L = Token<IO, D, HB>;
    constexpr int smem = sizeof(typename L::Smem);
    static_assert(smem <= 227 * 1024, "shared memory");
    static_assert(L::HALF % 1024 == 0 && offsetof(typename L::Smem, q) % 16 == 0 && offsetof(typename L::Smem, full) % 8 == 0, "alignment");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) { return cudaFuncSetAttribute(paged_token_kernel<IO, D, HB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    if (!encode_cache(&km, a.k, a, L::KEYS, L::SIZE) || !encode_cache(&vm, a.v, a, L::KEYS, L::SIZE)) return cudaErrorInvalidValue;
    TokenWork w;
    lay_out(w, a);
    e = launch_dependent(paged_token_kernel<IO, D, HB>, CTAS, L::THREADS, smem, st, a, w, km, vm);
    if (e == cudaSuccess) e = launch_dependent(token_join_kernel<IO, D, L::ROWS>, CTAS, 32 * std::min(L::ROWS, a.G), 0, st, a, w);
    return e;
}

template <int D> cudaError_t launch_heads(const PagedArgs& a, bool f32, cudaStream_t st)
{
    if (f32) return launch<float, D, 1>(a, st);
    return unit_rows(a) == 8 ? launch<__nv_bfloat16, D, 1>(a, st) : launch<__nv_bfloat16, D, 2>(a, st);
}

}  // namespace

// A unit holds the heads of a group up to these: more of them would read the cache again for each, and take the kernels for
// chunks, whose tiles hold up to 256 rows (64 sequences of 8192 tokens, four key heads of 32 query heads: 195 us there, 355 here).
bool paged_token_wanted(const PagedArgs& a, bool f32) { return a.G <= (f32 ? 8 : 16); }

size_t paged_token_workspace_bytes(const PagedArgs& a)
{
    TokenWork w;
    return lay_out(w, a);
}

cudaError_t launch_paged_token(const PagedArgs& a, bool f32, cudaStream_t st)
{
    switch (a.D) {
    case 32: return launch_heads<32>(a, f32, st);
    case 64: return launch_heads<64>(a, f32, st);
    case 128: return launch_heads<128>(a, f32, st);
    default: return launch_heads<256>(a, f32, st);
    }
}

}  // namespace kda
