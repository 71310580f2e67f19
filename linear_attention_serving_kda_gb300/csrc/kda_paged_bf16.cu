// kda_paged_bf16.cu -- attention of chunks of bf16 rows over a paged cache on the tensor cores.
//
// A CTA holds one or two tiles of 128 rows (tokens times the heads that share a key head) and goes through its
// tokens KEYS at a time:
//     S = Q K^T            tcgen05, Q and K from shared memory, S in TMEM
//     W = 2^(c S - m)      a thread a row: c = scale log2 e, m the row's running maximum of c S
//     O = O + W V          tcgen05, W (bf16) from TMEM where S lay, V from shared memory, O in TMEM
// m lags behind the true maximum by up to 2^8 (the weights stay within fp32 and bf16 by far), so
// that O is rarely rescaled; the sum of the weights is fp32, of the weights before their rounding.
// The two tiles' products and exponentials alternate: while one tile's scores are exponentiated, the tensor
// cores work for the other; with one tile, two steps of it do.
// The weights are rounded to bf16 (2^-8 of each at most, with either sign: their sum is off by less than the outputs' own rounding).
// What bounds it: for long chunks of heads of 128 the products, and the power that they draw.  8192 rows of 32 heads of 128 run
// at 1580 TFLOP/s without a mask (1540 when called without a pause), at 1440 with one; the library's plain product reaches 1908.  Heads of 64 do
// half the products a score and stop at 940 (860 with a mask), 16 heads of 256 at 1120: latency in both, no unit is full (64: tensor cores
// 36 % of their cycles, issue slots 46, exponential unit 37; 256: 47, 21, 12 and L2 37, where the one tile of rows of a CTA leaves a warpgroup
// idle and its steps stand one behind the other).  A unit costs some 10 us besides where prompts are short (64 prompts of 333 rows 193 us).
#include <cuda.h>

#include "kda_paged_plan.cuh"

namespace kda {
namespace {

using namespace paged;

constexpr int THREADS = 384;  // two softmax warpgroups, a warp that issues products, one that loads keys and values, two that load rows and store outputs
constexpr int CTAS = 152;  // one an SM
constexpr float LAG = 8.f;

template <int DP> struct Shape {
    static constexpr int TILES = DP == 256 ? 1 : 2;    // tiles of 128 rows: TMEM holds 512 columns, O takes DP of them a tile
    static constexpr int KEYS = DP == 256 ? 64 : 128;
    // Places of a unit besides its key tiles.  None to four, 32 heads of 128: a prompt of 8192 rows 515, 405, 383, 388, 394 us; eight of 4096
    // 935, 800, 793, 808, 823.  16 of 256: a prompt of 8192 rows 627, 546, 493, 495, 498.
    static constexpr int UNIT = DP == 256 ? 3 : 2;
    static constexpr int BLOCKS = DP / 64;             // 128-byte pieces of a row
    static constexpr int SLOT = KEYS * DP * 2;
    static constexpr int SLOTS = DP == 64 ? 8 : 5;
    static constexpr int Q = TILES * 128 * DP * 2;
    static constexpr int OUT = 128 * DP * 2 / SLOT;    // slots that a tile's outputs pass through, COLS channels in each
    static constexpr int COLS = SLOT / 256;
    struct Smem {
        unsigned char q[Q];
        unsigned char ring[SLOTS * SLOT];
        uint64_t full[SLOTS], empty[SLOTS], scores[2], weights[2], product[2], rows[2], free[2], taken[2], ready[2][2], drained;
        uint32_t hidden[8], tmem;
        int dead;  // a wait ran out
        Start start;
    };
};

// Shared-memory descriptors of operands in 128-byte rows with the 128-byte swizzle, lower words (the upper one is
// the same for all: eight rows are 1024 bytes).  A slice of 16 inner values lies 32 bytes on within 64 of them for rows along
// the inner dimension (Q, K), 16 rows on for rows along the outer one (V; `lead` bytes from 64 outer values to the next).
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_inner(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_outer(uint32_t saddr, uint32_t lead) { return (saddr >> 4) | ((lead >> 4) << 16); }

// D (TMEM) (+)= A B^T; one thread issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
        : "memory");
}

// The first lane's value, which the compiler then knows to be the warp's: operands of products come from uniform registers,
// and moving each one there by itself was most of the time that issuing them took.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void commit_to(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A place in the ring of SLOTS tiles and the parity of its use.
template <int SLOTS> struct Place {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void on(uint32_t n)
    {
        slot += n;
        if (slot >= SLOTS) {
            slot -= SLOTS;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(ptx::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, const void* src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x), "r"(y), "r"(z),
                 "r"(ptx::smem_u32(src))
                 : "memory");
}

// A tile's rows as whole tokens of all the group's heads: a box of the queries and of the output.
__host__ __device__ inline bool whole_tokens(int G) { return (G & (G - 1)) == 0 && G <= 128; }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// the n lowest bits, none for n <= 0, all for n >= 32
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Steps of a piece of a unit: with two tiles of rows, step s is tile s & 1 over key tile s >> 1; with one, key tile s.  Step
// s uses S's buffer s & 1.  Everyone counts the phases of every barrier alike from the pieces themselves.
struct Work : Walk {
    int tiles, count, steps, k0, k1;  // tiles of rows, key tiles, steps, tokens
    bool staged;                      // the outputs leave through slots of the ring
    __device__ __forceinline__ void derive(int keys)
    {
        tiles = rows > 128 ? 2 : 1;
        count = t1 - t0;
        steps = count * tiles;
        k0 = lo + t0 * keys;
        k1 = min(hi, lo + t1 * keys);
        staged = whole() && count > 0;
    }
};

template <int DP, int D> __global__ void __launch_bounds__(THREADS, 1)
paged_bf16_kernel(const PagedArgs a, const Plan p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap)
{
    using L = Shape<DP>;
    constexpr int KEYS = L::KEYS, BLOCKS = L::BLOCKS, SLOT = L::SLOT, SLOTS = L::SLOTS;
    extern __shared__ __align__(1024) unsigned char raw[];
    auto& s = *reinterpret_cast<typename L::Smem*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            ptx::mbar_init(&s.full[i], 1);
            ptx::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s.scores[i], 1);
            ptx::mbar_init(&s.product[i], 1);
            ptx::mbar_init(&s.weights[i], 4);
            ptx::mbar_init(&s.rows[i], whole_tokens(a.G) ? 1 : 2);
            ptx::mbar_init(&s.free[i], 1);
            ptx::mbar_init(&s.taken[i], 4);
            ptx::mbar_init(&s.ready[i][0], 4);
            ptx::mbar_init(&s.ready[i][1], 4);
        }
        s.dead = 0;
        ptx::mbar_init(&s.drained, 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (tid == 32) {  // the maps are the launch's own arguments: no need to wait for them
        ptx::prefetch_map(&kmap);
        ptx::prefetch_map(&vmap);
        ptx::prefetch_map(&qmap);
        ptx::prefetch_map(&omap);
    }
    if (warp == 8) ptx::tmem_alloc(&s.tmem, 512);
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns: they begin at 0 (a constant keeps the products' operands out of registers)
    ptx::grid_dependency_wait();
    find_start<THREADS / 32>(a, p, s.start);
    if (tid == 0) p.cut[blockIdx.x].rows = 0;
    // A wait that runs out ends its role's work (and with it, one by one, the others').  What the CTA has not written by then stays unwritten, by
    // the storing warps and by the join (PART_LOST): softmax warps that go on without waits arrive early at barriers that others of their tile share, so that nothing
    // behind those is sure.  They set `dead` before such an arrival; it is looked at after it.
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return ptx::mbar_wait(bar, parity & 1, a.polls); };
    // One that lasts a piece of a unit, of n key tiles: a poll that nothing ends lasts 3.7 us, a tile 1.3 (two tiles of 128 rows by 128 keys of 64), so that
    // PAGED_POLLS are 15 s, 12 million tiles; the limit grows with n from 2^16 of them on.
    const auto wait_unit = [&](uint64_t* bar, uint32_t parity, int n) { return ptx::mbar_wait(bar, parity & 1, a.unit_polls * (1 + ((uint32_t)n >> 16))); };
    const auto report = [&](bool ok) {
        if (!ok && lane == 0) flag_status(a.dev_status, KDA_DEV_TIMEOUT);
    };
    const auto dead = [&] { return *reinterpret_cast<volatile int*>(&s.dead) != 0; };
    constexpr uint32_t O0 = 256;  // S: columns 0 .. 2 KEYS - 1, O behind

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 9) {
            // ---- loads: keys and values in the order in which the products meet them
            uint32_t use = 0, kt = 0;
            bool ok = (int)blockIdx.x != a.stalled;
            const int box = min(KEYS, 1 << a.page_shift), boxes = KEYS / box;
            Work w;
            for (w.start(p, s.start); ok && w.step(a, p);) {
                if (!w.act) continue;
                w.derive(KEYS);
                const int ahead = w.tiles == 1 ? 2 : 1;
                const auto load = [&](const CUtensorMap* map, int j, bool keys) {
                    const int slot = use % SLOTS, t0 = w.k0 + j * KEYS, t = t0 + lane % boxes * box, blk = lane / boxes;
                    int page = 0;
                    const bool mine = blk < BLOCKS && t < w.k1;
                    if (mine) page = a.pages[(long long)w.seq * a.width + (t >> a.page_shift)];
                    const bool gone = mine && (page < 0 || page >= a.num_pages);
                    const uint32_t all = __ballot_sync(0xffffffffu, mine);
                    uint32_t hide = __ballot_sync(0xffffffffu, gone && blk == 0);
                    if (!(ok = wait(&s.empty[slot], (use / SLOTS) & 1 ^ 1))) return;
                    if (lane == 0) {
                        if (keys) {
                            s.hidden[kt & 7] = hide;
                            if (hide) flag_status(a.dev_status, KDA_DEV_BAD_PAGE);
                        }
                        ptx::mbar_arrive_expect_tx(&s.full[slot], __popc(all) * box * 128);
                    }
                    __syncwarp();
                    if (mine) {
                        unsigned char* dst = s.ring + slot * SLOT + blk * (KEYS * 128) + lane % boxes * box * 128;
                        tma_load_4d(dst, map, blk * 64, t & ((1 << a.page_shift) - 1), w.head, gone ? -1 : page, &s.full[slot]);
                    }
                    if (keys) ++kt;
                    ++use;
                };
                for (int j = 0; j < min(ahead, w.count) && ok; ++j) load(&kmap, j, true);
                for (int j = 0; j < w.count && ok; ++j) {
                    load(&vmap, j, false);
                    if (ok && j + ahead < w.count) load(&kmap, j + ahead, true);
                }
                if (w.staged)  // slots for the outputs
                    for (int i = 0; i < w.tiles * L::OUT && ok; ++i, ++use) {
                        if (!(ok = wait(&s.empty[use % SLOTS], use / SLOTS + 1))) break;
                        if (lane == 0) ptx::mbar_arrive(&s.full[use % SLOTS]);
                    }
            }
            report(ok);
            // what is on its way has to land first (it has, unless those who wait for it gave up)
            for (uint32_t u = use > SLOTS ? use - SLOTS : 0; u < use; ++u) ptx::mbar_wait(&s.full[u % SLOTS], (u / SLOTS) & 1, PAGED_POLLS);
        } else if (warp >= 10) {
            // ---- rows: a tensor copy, or (tiles that cut tokens) half of each tile by either warp, 16-byte pieces permuted within
            // eight rows as the descriptor expects; and the outputs of the unit before from the ring's slots, the first slot by one warp,
            // the second by the other.  (Outputs of units in turn are announced on two barriers: with one, softmax warps that are through with the next unit
            // before this warp looks for the one before would make two uses look like none.  They cannot be through with the one after that: its rows come from this
            // warp, behind its stores, or (second slot, rows by the other warp) its slot lies two units, eight places of the ring at least, behind this one's.)  (Pieces by threads take 3 us a unit, copies nothing that shows: 64 prompts of 333 rows 202 us with them, 190 with copies.)
            static_assert(SLOTS <= 8, "two units use the whole ring");
            constexpr int PIECES = DP / 8, AT_ONCE = 32 / PIECES;  // rows that a warp's 32 pieces make
            const int me = warp & 1, e = lane % PIECES, r0 = me * 64 + lane / PIECES;
            const int dt = group_of(a, AT_ONCE), dg = AT_ONCE - dt * a.G;
            uint32_t count[2] = {0, 0}, stored = 0, use = 0;
            int before = 0;  // key tiles of the piece before
            bool ok = true;
            // slot `me` of a unit that leaves through the ring
            struct {
                bool any = false;
                int begin, row0, rows, head, count;
                uint32_t use;
            } out;
            const auto store = [&] {
                if (!out.any || !ok) return;
                out.any = false;
                constexpr int COLS = L::COLS, PC = COLS / 8, ROWS_AT_ONCE = 32 / PC;
                const int t = L::OUT == 1 ? me : 0, col = L::OUT == 1 ? 0 : me * COLS, c8 = lane % PC;
                ok = wait_unit(&s.ready[me][stored & 1], stored >> 1, out.count);
                ++stored;
                if (!(ok = !__any_sync(0xffffffffu, !ok || dead()))) return;
                const unsigned char* slot = s.ring + out.use % SLOTS * SLOT;
                const int last = min(128, out.rows - t * 128);
                if (last == 128 && whole_tokens(a.G)) {
                    if (lane == 0) {
                        for (int b = 0; b < COLS / 64; ++b)
                            tma_store_3d(&omap, col + b * 64, out.head * a.G, out.begin + group_of(a, out.row0 + t * 128), slot + b * (128 * 128));
                        ptx::bulk_commit();
                        ptx::bulk_wait_read_all();
                        ptx::mbar_arrive(&s.empty[out.use % SLOTS]);
                    }
                    __syncwarp();
                    return;
                }
                const int ot = group_of(a, ROWS_AT_ONCE), og = ROWS_AT_ONCE - ot * a.G, f0 = out.row0 + t * 128 + lane / PC, tok0 = group_of(a, f0);
                int g = f0 - tok0 * a.G;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + ((size_t)(out.begin + tok0) * a.Hq + out.head * a.G) * D + col + c8 * 8;
#pragma unroll 8
                for (int rr = lane / PC; rr < last; rr += ROWS_AT_ONCE) {
                    const uint4 x = *reinterpret_cast<const uint4*>(slot + c8 / 8 * (128 * 128) + rr * 128 + ((c8 ^ rr) & 7) * 16);
                    if (col + c8 * 8 < D) *reinterpret_cast<uint4*>(dst + (size_t)g * D) = x;
                    g += og;
                    dst += (size_t)ot * a.Hq * D;
                    if (g >= a.G) {
                        g -= a.G;
                        dst += (size_t)a.Hq * D;
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s.empty[out.use % SLOTS]);
            };
            Work w;
            for (w.start(p, s.start); ok && w.step(a, p);) {
                if (!w.act || w.n == 0) continue;
                w.derive(KEYS);
#pragma unroll
                for (int t = 0; t < L::TILES; ++t) {
                    if (t >= w.tiles || (whole_tokens(a.G) && me == 1)) break;
                    if (!(ok = wait_unit(&s.free[t], count[t] + 1, before))) break;  // the scores of the unit before are done
                    ++count[t];
                    unsigned char* base = s.q + t * (128 * DP * 2);
                    if (whole_tokens(a.G)) {
                        if (lane == 0) {
                            ptx::mbar_arrive_expect_tx(&s.rows[t], 128 * DP * 2);
                            for (int b = 0; b < BLOCKS; ++b)
                                tma_load_3d(base + b * (128 * 128), &qmap, b * 64, w.head * a.G, w.begin + group_of(a, w.row0 + t * 128), &s.rows[t]);
                        }
                        __syncwarp();
                        continue;
                    }
                    const int f = w.row0 + t * 128 + r0, tok = group_of(a, f);
                    int g = f - tok * a.G;
                    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (w.begin + tok) * a.q_stride + (long long)w.head * a.G * D + e * 8;
                    unsigned char* dst = base + e / 8 * (128 * 128);
#pragma unroll 4
                    for (int r = r0; r < r0 / 64 * 64 + 64; r += AT_ONCE) {
                        const bool in = t * 128 + r < w.rows && e * 8 < D;
                        ptx::cp_async16(dst + r * 128 + ((e % 8) ^ (r & 7)) * 16, in ? q + (long long)g * D : static_cast<const __nv_bfloat16*>(a.q), in ? 16 : 0);
                        g += dg;
                        q += dt * a.q_stride;
                        if (g >= a.G) {
                            g -= a.G;
                            q += a.q_stride;
                        }
                    }
                    ptx::cp_async_commit();
                    ptx::cp_async_wait_all();
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&s.rows[t]);
                }
                before = w.count;
                store();  // of the unit before: these rows went first
                use += 2 * w.count;
                if (w.staged) {
                    out.any = me < w.tiles * L::OUT;
                    out.begin = w.begin;
                    out.row0 = w.row0;
                    out.rows = w.rows;
                    out.head = w.head;
                    out.count = w.count;
                    out.use = use + me;
                    use += w.tiles * L::OUT;
                }
            }
            store();
            report(ok);
            ptx::bulk_wait_all();
            // what is on its way has to land first (as above)
            if (whole_tokens(a.G) && me == 0)
                for (int t = 0; t < L::TILES; ++t)
                    if (count[t]) ptx::mbar_wait(&s.rows[t], (count[t] - 1) & 1, PAGED_POLLS);
        } else if (warp == 8) {
            // ---- products
            const bool leader = ptx::elect_one();
            constexpr uint32_t ID_S = ptx::idesc_bf16(128, KEYS), ID_O = ptx::idesc_bf16(128, DP) | (1u << 16);  // V: inner dimension by rows
            constexpr uint32_t STEP = SLOT / 16;
            const uint32_t qd = desc_inner(ptx::smem_u32(s.q)), kd = desc_inner(ptx::smem_u32(s.ring)),
                           vd = desc_outer(ptx::smem_u32(s.ring), KEYS * 128);
            Place<SLOTS> first;
            uint32_t wcount[2] = {0, 0}, qcount[2] = {0, 0};
            bool ok = true;
            Work w;
            for (w.start(p, s.start); ok && w.step(a, p);) {
                if (!w.act || w.n == 0) continue;
                w.derive(KEYS);
                const bool two = w.tiles == 2;
                // the ring holds K0 (K1, with one tile) V0 K1 (K2) V1 ...
                Place<SLOTS> kp = first, vp = first;
                vp.on(two ? 1 : min(2, w.count));
                // scores of row tile t over the keys at kp into buffer b, products of the weights there with the values at vp: by the leader.
                // Between a tile's weights and its next scores nothing is waited for: every instruction there is time without products.
                uint32_t db, ebar, dv, vbar;  // operands and barriers of the slots at kp and vp
                const auto at_keys = [&] {
                    db = uniform(kd + kp.slot * STEP);
                    ebar = uniform(ptx::smem_u32(&s.empty[kp.slot]));
                };
                const auto at_values = [&] {
                    dv = uniform(vd + vp.slot * STEP);
                    vbar = uniform(ptx::smem_u32(&s.empty[vp.slot]));
                };
                const auto scores = [&](int t, int b) {
                    const uint32_t da = qd + t * (128 * DP * 2 / 16);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        mma_ss(tmem + b * KEYS, da + ((k / 4) * (128 * 128) + (k % 4) * 32) / 16, db + ((k / 4) * (KEYS * 128) + (k % 4) * 32) / 16, ID_S, k > 0);
                    ptx::mma_commit(&s.scores[b]);
                };
                const auto values = [&](int t, int b, int j) {
#pragma unroll
                    for (int k = 0; k < KEYS / 16; ++k)
                        mma_ts(tmem + O0 + t * DP, tmem + b * KEYS + k * 8, dv + k * 2048 / 16, ID_O, k > 0 || j > 0);
                };
                const auto values_here = [&](int j) {
                    if (!wait(&s.full[vp.slot], vp.phase)) return false;
                    const int have = w.k1 - w.k0 - j * KEYS, from = w.seen - w.k0 - j * KEYS;
                    if (have < KEYS || from > 0) {  // what lies behind the tokens, or before the window, may be anything: zeros, whose weights are zero
                        // (a linear fill of each block's last rows: with a division a piece it took 5500 cycles, the next unit's start)
#pragma unroll
                        for (int blk = 0; blk < BLOCKS; ++blk) {
                            unsigned char* v = s.ring + vp.slot * SLOT + blk * (KEYS * 128);
                            for (int at = have * 128 + lane * 16; at < KEYS * 128; at += 512) *reinterpret_cast<uint4*>(v + at) = make_uint4(0, 0, 0, 0);
                            for (int at = lane * 16; at < from * 128; at += 512) *reinterpret_cast<uint4*>(v + at) = make_uint4(0, 0, 0, 0);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    return true;
                };
                at_keys();
                if (two) {
                    ok = wait(&s.full[kp.slot], kp.phase) && wait(&s.rows[0], qcount[0]);
                    if (ok && leader) scores(0, 0);
                    __syncwarp();
                    ok = ok && wait(&s.rows[1], qcount[1]);
                    if (ok && leader) {
                        scores(1, 1);
                        commit_to(ebar);
                        if (w.count == 1) {
                            ptx::mma_commit(&s.free[0]);
                            ptx::mma_commit(&s.free[1]);
                        }
                    }
                    __syncwarp();
                    kp.on(2);
                    for (int j = 0; j < w.count && ok; ++j) {
                        const bool more = j + 1 < w.count;
                        at_keys();
                        at_values();
                        ok = values_here(j) && (!more || wait(&s.full[kp.slot], kp.phase));
                        if (j == 0) ok = ok && wait(&s.taken[0], qcount[0] + 1) && wait(&s.taken[1], qcount[1] + 1);  // O of the unit before is read
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            ok = ok && wait(&s.weights[t], wcount[t]);
                            ++wcount[t];
                            ptx::tc_fence_after();
                            if (ok && leader) {
                                values(t, t, j);
                                if (t == 1) commit_to(vbar);
                                if (more) {
                                    scores(t, t);
                                    if (t == 1) commit_to(ebar);
                                    if (j + 2 == w.count) ptx::mma_commit(&s.free[t]);
                                } else {
                                    ptx::mma_commit(&s.product[t]);
                                }
                            }
                            __syncwarp();
                        }
                        kp.on(2);
                        vp.on(2);
                    }
                } else {
                    ok = wait(&s.rows[0], qcount[0]);
                    for (int j = 0; j < min(2, w.count) && ok; ++j) {
                        at_keys();
                        ok = wait(&s.full[kp.slot], kp.phase);
                        if (ok && leader) {
                            scores(0, j);
                            commit_to(ebar);
                            if (j + 1 == w.count) ptx::mma_commit(&s.free[0]);
                        }
                        __syncwarp();
                        kp.on(j == 0 ? 1 : 2);
                    }
                    for (int j = 0; j < w.count && ok; ++j) {
                        const bool more = j + 2 < w.count;
                        const int b = j & 1;
                        at_keys();
                        at_values();
                        ok = values_here(j);
                        // O of the unit before is read, also its second tile's, if it had one (else of the last that had): product[1] is about to be used again, and whoever
                        // still waits for its last use would take two for none
                        if (j == 0) ok = ok && wait(&s.taken[0], qcount[0] + 1) && (L::TILES == 1 || wait(&s.taken[1], qcount[1] + 1));
                        const bool there = __all_sync(0xffffffffu, more && ptx::mbar_test(&s.full[kp.slot], kp.phase));
                        ok = ok && wait(&s.weights[b], b ? wcount[1]++ : wcount[0]++);
                        ptx::tc_fence_after();
                        const auto next = [&] {
                            scores(0, b);
                            commit_to(ebar);
                            if (j + 3 == w.count) ptx::mma_commit(&s.free[0]);
                        };
                        if (ok && leader) {
                            values(0, b, j);
                            ptx::mma_commit(&s.product[b]);
                            commit_to(vbar);
                            if (there) next();
                        }
                        __syncwarp();
                        if (more && !there) {  // keys that are not there yet do not hold up the product
                            ok = ok && wait(&s.full[kp.slot], kp.phase);
                            if (ok && leader) next();
                            __syncwarp();
                        }
                        kp.on(2);
                        vp.on(j == w.count - 2 ? 1 : 2);
                    }
                }
                const uint32_t end = first.slot + 2 * w.count + (w.staged ? w.tiles * L::OUT : 0);
                first.slot = end % SLOTS;
                first.phase ^= end / SLOTS & 1;
                ++qcount[0];
                qcount[1] += two;
            }
            report(ok);
            // nothing may be on its way when TMEM is freed
            if (leader) ptx::mma_commit(&s.drained);
            __syncwarp();
            ptx::mbar_wait(&s.drained, 0, PAGED_POLLS);
        }
    } else {
        // ---- a thread a row: exponentials, rescaling, outputs.  (After a wait that ran out a warp goes on without waits
        // and outputs, so that it still meets the others at the barriers.)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2, r = tid & 127;  // tile, row of it
        const uint32_t tl = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const float c = a.scale * 1.4426950408889634f;
        uint32_t scount[2] = {0, 0}, sbase[2] = {0, 0}, pcount[2] = {0, 0}, kt = 0, use = 0, staged = 0;
        bool ok = true;
        Work w;
        for (w.start(p, s.start); w.step(a, p);) {
            if (t >= L::TILES) break;
            if (!w.act) continue;
            w.derive(KEYS);
            const int row = t * 128 + r;
            const bool mine = t < w.tiles;
            const bool live = mine && t * 128 + (warp & 3) * 32 < w.rows;  // the warp has rows
            const int f = w.row0 + min(row, w.rows - 1), tok = group_of(a, f), head = w.head * a.G + f - tok * a.G;
            float m = -INFINITY, sum = 0.f;
            if (mine && w.count > 0) {
                const int pos = w.pos0() + tok;
                const int hi = a.causal ? min(w.k1, pos + 1) : w.k1;
                const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
                for (int st = w.tiles == 2 ? t : 0; st < w.steps; st += w.tiles) {
                    const int j = w.tiles == 2 ? st >> 1 : st, b = st & 1, k0 = w.k0 + j * KEYS;
                    ok = ok && wait(&s.scores[b], scount[b]);
                    ++scount[b];
                    ptx::tc_fence_after();
                    if (live && ok) {
                        // 64 scores at a time: the first ones' maximum while the second ones come
                        float v[KEYS], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        auto& v0 = *reinterpret_cast<float(*)[64]>(v);
                        auto& v1 = *reinterpret_cast<float(*)[64]>(v + (KEYS - 64));
                        const uint32_t hide = *reinterpret_cast<volatile uint32_t*>(&s.hidden[(kt + j) & 7]);
                        const bool masked = __any_sync(0xffffffffu, k0 + KEYS > hi || k0 < lo) || hide;
                        const int box_shift = min(a.page_shift, KEYS == 128 ? 7 : 6);
                        const auto look = [&](int from) {
                            if (masked)
#pragma unroll
                                for (int i = from; i < from + 64; i += 32) {
                                    uint32_t seen = low_bits(hi - k0 - i) & ~low_bits(lo - k0 - i);
                                    if ((hide >> (i >> box_shift)) & 1) seen &= 0xffff0000u;
                                    if ((hide >> ((i + 16) >> box_shift)) & 1) seen &= 0x0000ffffu;
                                    if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
                                    for (int e = 0; e < 32; ++e) v[i + e] = (seen >> e) & 1 ? v[i + e] : -INFINITY;
                                }
#pragma unroll
                            for (int i = from; i < from + 64; i += 8)
#pragma unroll
                                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], v[i + 2 * e], v[i + 2 * e + 1]);
                        };
                        ptx::tmem_ld64_async(tl + b * KEYS, v0);
                        ptx::tmem_wait_ld64(v0);
                        if constexpr (KEYS == 128) ptx::tmem_ld64_async(tl + b * KEYS + 64, v1);
                        look(0);
                        if constexpr (KEYS == 128) {
                            ptx::tmem_wait_ld64(v1);
                            look(64);
                        }
                        const float most = c * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        const bool grow = most > m + LAG || (m == -INFINITY && most > m);
                        if (__any_sync(0xffffffffu, grow)) {
                            const float next = grow ? most : m, fac = grow ? exp2_sfu(m - next) : 1.f;
                            sum *= fac;
                            if (j > 0) {
                                // with one tile the step before's product may still run (with two it had to end before these scores began)
                                if (w.tiles == 1) ok = wait(&s.product[b ^ 1], pcount[b ^ 1] + (st - 1) / 2);
                                ptx::tc_fence_after();
#pragma unroll 1
                                for (int e = 0; e < DP; e += 32) {
                                    float o[32];
                                    ptx::tmem_ld32(tl + O0 + t * DP + e, o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] *= fac;
                                    ptx::tmem_st32(tl + O0 + t * DP + e, o);
                                }
                            }
                            m = next;
                        }
                        const float2 c2 = both2(c), base = both2(m == -INFINITY ? 0.f : -m);
                        float2 part[2] = {both2(0.f), both2(0.f)};
#pragma unroll
                        for (int i = 0; i < KEYS; i += 32) {
                            uint32_t packed[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 y = fma2(make_float2(v[i + 2 * e], v[i + 2 * e + 1]), c2, base);
                                y.x = exp2_sfu(y.x);
                                y.y = exp2_sfu(y.y);
                                part[e & 1] = add2(part[e & 1], y);
                                packed[e] = pack_bf16(y.x, y.y);
                            }
                            ptx::tmem_st16_async(tl + b * KEYS + i / 2, packed);
                        }
                        part[0] = add2(part[0], part[1]);
                        sum += part[0].x + part[0].y;
                        ptx::tmem_wait_st();
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (!ok) *reinterpret_cast<volatile int*>(&s.dead) = 1;
                        ptx::mbar_arrive(&s.weights[b]);
                    }
                }
            }
            kt += w.count;
            if (mine) {
                if (w.count > 0) {
                    const int last = w.steps - 1, b = w.tiles == 2 ? t : last & 1;
                    ok = ok && wait(&s.product[b], w.tiles == 2 ? pcount[b] : pcount[b] + last / 2);
                    if (!ok) *reinterpret_cast<volatile int*>(&s.dead) = 1;
                    ptx::tc_fence_after();
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const size_t cell = (size_t)blockIdx.x * 2 + (w.t0 == 0);
                if (w.staged) {
                    // a thread's row into the slot, 16-byte pieces permuted within eight rows; whole rows leave from there
                    use += 2 * w.count + t * L::OUT;
                    constexpr int COLS = L::COLS;
#pragma unroll 1
                    for (int i = 0; i < L::OUT; ++i, ++use) {
                        unsigned char* slot = s.ring + use % SLOTS * SLOT;
                        ok = ok && wait(&s.full[use % SLOTS], use / SLOTS);
                        if (!ok) *reinterpret_cast<volatile int*>(&s.dead) = 1;
                        if (live && ok) {
#pragma unroll 1
                            for (int e = 0; e < COLS; e += 32) {
                                float o[32];
                                ptx::tmem_ld32(tl + O0 + t * DP + i * COLS + e, o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = sum == 0.f ? 0.f : o[k] * inv;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    *reinterpret_cast<uint4*>(slot + e / 64 * (128 * 128) + r * 128 + ((e % 64 / 8 + k) ^ (r & 7)) * 16) =
                                        make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                                   pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
                            }
                        }
                        ptx::tc_fence_before();
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (i == L::OUT - 1) ptx::mbar_arrive(&s.taken[t]);  // O may be overwritten
                            ptx::mbar_arrive(&s.ready[L::OUT == 1 ? t : i][staged & 1]);
                        }
                    }
                    use += (w.tiles - 1 - t) * L::OUT;
                    ++staged;
                } else {
                    if (live) {
#pragma unroll 1
                        for (int e = 0; e < D; e += 32) {
                            float o[32];
                            if (w.count > 0) {
                                ptx::tmem_ld32(tl + O0 + t * DP + e, o);
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = 0.f;
                            }
                            if (row >= w.rows || !ok) continue;
                            if (w.count > 0) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    p.o[(cell * (D / 4) + e / 4 + i) * p.part_rows + row] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            } else {  // rows that see nothing
                                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((size_t)(w.begin + tok) * a.Hq + head) * D + e);
#pragma unroll
                                for (int i = 0; i < 4; ++i) dst[i] = make_uint4(0, 0, 0, 0);
                            }
                        }
                    }
                    if (w.count > 0) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&s.taken[t]);
                        use += 2 * w.count;
                    }
                }
                ok = !__any_sync(0xffffffffu, !ok || dead());
                if (live && row < w.rows) {
                    if (!w.whole()) p.ml[cell * p.part_rows + row] = make_float2(m, ok ? sum : PART_LOST);
                    else if (a.lse && ok) a.lse[(size_t)(w.begin + tok) * a.Hq + head] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
                }
            } else {
                use += 2 * w.count + (w.staged ? w.tiles * L::OUT : 0);
            }
            if (tid == 0 && w.t0 == 0 && !w.whole())
                p.cut[blockIdx.x] = {s.start.line, w.begin, w.row0, w.rows, w.head, owner(s.start.line, w.end(p) - 1, p.ctas)};
            for (int b = 0; b < 2; ++b) {
                scount[b] = sbase[b] += w.tiles == 2 ? w.count : (w.count + 1 - b) / 2;
                pcount[b] += w.tiles == 2 ? min(w.count, 1) : (w.count + 1 - b) / 2;
            }
            // the other warpgroup, without rows in this item, may not run ahead over phases of barriers that it did not wait for
            if (L::TILES == 2 && w.tiles == 1) {
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
        }
        report(ok);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 8) ptx::tmem_dealloc(tmem, 512);
}

// [num_pages][Hkv][page_size][D] by the cache's strides; boxes of a page's (or a tile's) tokens and 64 channels of one head.
bool encode_cache(CUtensorMap* m, const void* base, const PagedArgs& a, int keys)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t P = (cuuint64_t)1 << a.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, P, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.token_stride * 2, (cuuint64_t)a.head_stride * 2, (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min<cuuint64_t>(P, keys), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T][Hq][D] rows; boxes of 128 / G tokens of a group's heads and 64 channels.
bool encode_rows(CUtensorMap* m, const void* base, long long stride, const PagedArgs& a)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)stride * 2};
    const int G = whole_tokens(a.G) ? a.G : 1;  // (not used otherwise)
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int D> cudaError_t launch(const PagedArgs& a, cudaStream_t st)
{
    using L = Shape<DP>;
    constexpr int smem = sizeof(typename L::Smem);
    static_assert(smem <= 227 * 1024, "shared memory");
    static_assert(offsetof(typename L::Smem, ring) % 1024 == 0 && L::SLOT % 1024 == 0 && offsetof(typename L::Smem, full) % 8 == 0, "alignment");
    static PerDeviceOnce once;
    cudaError_t e = once.run([](int) {
        return cudaFuncSetAttribute(paged_bf16_kernel<DP, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm, qm, om;
    if (!encode_cache(&km, a.k, a, L::KEYS) || !encode_cache(&vm, a.v, a, L::KEYS) ||
        !encode_rows(&qm, a.q, a.q_stride, a) || !encode_rows(&om, a.out, (long long)a.Hq * a.D, a))
        return cudaErrorInvalidValue;
    Plan p;
    lay_out(p, a, 128 * L::TILES, L::KEYS, CTAS, L::UNIT);
    e = launch_dependent(paged_bf16_kernel<DP, D>, CTAS, THREADS, smem, st, a, p, km, vm, qm, om);
    if (e == cudaSuccess) e = launch_join<__nv_bfloat16, D>(a, p, st);
    return e;
}

}  // namespace

size_t paged_bf16_workspace_bytes(const PagedArgs& a)
{
    Plan p;
    return a.D == 256 ? lay_out(p, a, 128, 64, CTAS, 0) : lay_out(p, a, 256, 128, CTAS, 0);
}

cudaError_t launch_paged_bf16(const PagedArgs& a, cudaStream_t st)
{
    switch (a.D) {
    case 32: return launch<64, 32>(a, st);
    case 64: return launch<64, 64>(a, st);
    case 128: return launch<128, 128>(a, st);
    default: return launch<256, 256>(a, st);
    }
}

}  // namespace kda
