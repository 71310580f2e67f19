// kda_slots.cu -- forking, compacting and freeing the slots of a state pool.
//
// Pure data movement: a copied slot is read once and written once, so the
// bound is HBM bandwidth.  A fork's source is read once for each RUN of targets, from
// HBM once: seven copies of 24 layers of 2 MiB 70 us, 5.7 TB/s of what the copy has to move.
// 66 moves of 24 layers of 48 KiB with their plan 30 us, 5.1 TB/s, seven of the 30 the plan and the second launch.
#include "kda_check.h"
#include "kda_common.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int ST = 256;             // threads of a CTA
constexpr int PIECE = ST * 4 * 16;  // bytes one CTA moves at a time
constexpr int LIST = 2048;          // pairs kept in shared memory at a time
constexpr int RUN = 4;              // neighbouring pairs a CTA takes with a piece: a forked source is read once for them

__device__ __forceinline__ bool test_bit(const uint32_t* m, int i) { return (m[i >> 5] >> (i & 31)) & 1u; }
__device__ __forceinline__ void set_bit(uint32_t* m, int i) { atomicOr(m + (i >> 5), 1u << (i & 31)); }

// Collects the usable ones of pairs i0 .. i0 + LIST - 1 in `list`, in their
// order, so that every CTA comes to the same list.  keep(i, pair) says whether
// pair i is used.
template <class F> __device__ int collect(int i0, int n, int2* list, int* warp_tot, F&& keep)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, end = min(LIST, n - i0);
    int have = 0;
    for (int i = 0; i < end; i += ST) {
        int2 pr = make_int2(0, 0);
        const bool use = i + tid < end && keep(i0 + i + tid, pr);
        const uint32_t m = __ballot_sync(0xffffffffu, use);
        if (lane == 0) warp_tot[warp] = __popc(m);
        __syncthreads();
        int before = have;
        for (int w = 0; w < ST / 32; ++w) {
            if (w < warp) before += warp_tot[w];
            have += warp_tot[w];
        }
        if (use) list[before + __popc(m & ((1u << lane) - 1u))] = pr;
        __syncthreads();
    }
    return have;
}

struct PoolArgs {
    char* pool;
    long long layer_stride, slot_bytes;
    int layers, num_slots, n;
    const int32_t* src;
    const int32_t* dst;
    int32_t* dev_status;
};

// Items are (layer, piece of the slot, run of pairs) with the runs running
// fastest: neighbouring CTAs read the same piece of a forked source at about
// the same time, so it leaves HBM once.
__global__ void __launch_bounds__(ST) slots_copy_kernel(const PoolArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    extern __shared__ uint32_t maps[];  // three bit maps over the slots
    __shared__ int2 list[LIST];
    __shared__ int warp_tot[ST / 32];
    const int tid = threadIdx.x, words = (a.num_slots + 31) / 32;
    uint32_t *once = maps, *twice = maps + words, *source = maps + 2 * words;
    for (int i = tid; i < 3 * words; i += ST) maps[i] = 0;
    __syncthreads();
    bool bad = false;
    for (long long i = tid; i < a.n; i += ST) {
        const int s = a.src[i], d = a.dst[i];
        if (s < 0 || d < 0) continue;
        if (s >= a.num_slots || d >= a.num_slots) {
            bad = true;
            continue;
        }
        if (s == d) continue;
        const uint32_t bit = 1u << (d & 31);
        if (atomicOr(once + (d >> 5), bit) & bit) set_bit(twice, d);
        set_bit(source, s);
    }
    __syncthreads();
    const long long pieces = (a.slot_bytes + PIECE - 1) / PIECE;
    for (long long i0 = 0; i0 < a.n; i0 += LIST) {
        const int have = collect((int)i0, a.n, list, warp_tot, [&](int i, int2& pr) {
            const int s = a.src[i], d = a.dst[i];
            if (s < 0 || d < 0 || s >= a.num_slots || d >= a.num_slots || s == d) return false;
            if (test_bit(twice, d) || test_bit(source, d)) {
                bad = true;
                return false;
            }
            pr = make_int2(s, d);
            return true;
        });
        const int runs = (have + RUN - 1) / RUN;
        const long long items = pieces * a.layers * runs;
        for (long long w = blockIdx.x; w < items; w += gridDim.x) {
            const int first = (int)(w % runs) * RUN, last = min(first + RUN, have);
            const long long rest = w / runs;
            char* base = a.pool + (rest / pieces) * a.layer_stride;
            const long long off = (rest % pieces) * PIECE + tid * 16;
            uint4 v[4];
            int held = -1;
            for (int i = first; i < last; ++i) {
                const int2 pr = list[i];
                if (pr.x != held) {
                    const char* s = base + pr.x * a.slot_bytes + off;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (off + j * ST * 16 < a.slot_bytes) v[j] = *reinterpret_cast<const uint4*>(s + j * ST * 16);
                    held = pr.x;
                }
                char* d = base + pr.y * a.slot_bytes + off;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (off + j * ST * 16 < a.slot_bytes) *reinterpret_cast<uint4*>(d + j * ST * 16) = v[j];
            }
        }
        __syncthreads();
    }
    if (bad && blockIdx.x == 0) flag_status(a.dev_status, KDA_DEV_BAD_SLOT);
}

__global__ void __launch_bounds__(ST) slots_zero_kernel(const PoolArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ int2 list[LIST];
    __shared__ int warp_tot[ST / 32];
    const int tid = threadIdx.x;
    bool bad = false;
    const long long pieces = (a.slot_bytes + PIECE - 1) / PIECE;
    for (long long i0 = 0; i0 < a.n; i0 += LIST) {
        const int have = collect((int)i0, a.n, list, warp_tot, [&](int i, int2& pr) {
            const int d = a.dst[i];
            if (d >= a.num_slots) bad = true;
            pr = make_int2(d, d);
            return d >= 0 && d < a.num_slots;
        });
        const long long items = pieces * a.layers * have;
        for (long long w = blockIdx.x; w < items; w += gridDim.x) {
            const long long rest = w / have;
            char* d = a.pool + (rest / pieces) * a.layer_stride + list[w % have].y * a.slot_bytes;
            const long long off = (rest % pieces) * PIECE + tid * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (off + j * ST * 16 < a.slot_bytes)
                    *reinterpret_cast<uint4*>(d + off + j * ST * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    }
    if (bad && blockIdx.x == 0) flag_status(a.dev_status, KDA_DEV_BAD_SLOT);
}

// One CTA: counts the live slots, then ranks the holes below and the live
// slots above that count, a thousand slots at a time.
constexpr int PT = 1024;
__global__ void __launch_bounds__(PT) compact_plan_kernel(int S, const int32_t* live, int32_t* src, int32_t* dst,
                                                          int32_t* remap)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ int holes[PT / 32], movers[PT / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int L = 0;
    for (int i = 0; i < S; i += PT) L += __syncthreads_count(i + tid < S && live[i + tid] != 0);
    int nh = 0, nm = 0;
    for (int i = 0; i < S; i += PT) {
        const int at = i + tid;
        const bool in = at < S, lv = in && live[at] != 0;
        const bool hole = in && !lv && at < L, mover = lv && at >= L;
        const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
        if (lane == 0) {
            holes[warp] = __popc(mh);
            movers[warp] = __popc(mm);
        }
        __syncthreads();
        int h = nh, m = nm;
        for (int w = 0; w < PT / 32; ++w) {
            if (w < warp) {
                h += holes[w];
                m += movers[w];
            }
            nh += holes[w];
            nm += movers[w];
        }
        const uint32_t below = (1u << lane) - 1u;
        if (hole) dst[h + __popc(mh & below)] = at;
        if (mover) src[m + __popc(mm & below)] = at;
        if (in && !mover) remap[at] = lv ? at : -1;
        __syncthreads();
    }
    // as many holes below L as live slots above it: nh == nm
    for (int i = tid; i < S; i += PT) {
        if (i < nm) remap[src[i]] = dst[i];
        else src[i] = dst[i] = -1;
    }
}

int check_pool(const kda_slot_pool* p)
{
    if (!p || !p->pool || !aligned16(p->pool)) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_layers < 1 || p->num_slots < 1 || p->num_slots > KDA_MAX_POOL_SLOTS) return KDA_ERR_INVALID_ARGUMENT;
    if (p->slot_bytes <= 0 || p->slot_bytes % 16 != 0 || p->slot_bytes > INT64_MAX / p->num_slots)
        return KDA_ERR_INVALID_ARGUMENT;
    if (p->layer_stride_bytes % 16 != 0 || p->layer_stride_bytes < p->slot_bytes * p->num_slots ||
        p->layer_stride_bytes > INT64_MAX / p->num_layers)
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

PoolArgs pool_args(const kda_slot_pool* p, int32_t n, const int32_t* src, const int32_t* dst, int32_t* dev_status)
{
    PoolArgs a;
    a.pool = static_cast<char*>(p->pool);
    a.layer_stride = p->layer_stride_bytes;
    a.slot_bytes = p->slot_bytes;
    a.layers = p->num_layers;
    a.num_slots = p->num_slots;
    a.n = n;
    a.src = src;
    a.dst = dst;
    a.dev_status = dev_status;
    return a;
}

// One CTA per piece, up to eight on every SM.
int pool_grid(const kda_slot_pool* p, int32_t n)
{
    const double items = (double)((p->slot_bytes + PIECE - 1) / PIECE) * p->num_layers * n;
    return (int)std::max(1.0, std::min(items, 8.0 * sm_count()));
}

// The pool's bytes from its first slot to its last.
size_t pool_bytes(const kda_slot_pool* p)
{
    return (size_t)(p->num_layers - 1) * p->layer_stride_bytes + (size_t)p->num_slots * p->slot_bytes;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

KDA_API int kda_slots_copy(const kda_slot_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                           int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_pool(pool);
    if (rc != KDA_OK) return rc;
    if (n < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (n == 0) return KDA_OK;
    if ((rc = check_ptrs({src, dst})) != KDA_OK) return rc;
    const size_t all = pool_bytes(pool), ib = sizeof(int32_t) * (size_t)n;
    if (overlap(pool->pool, all, src, ib) || overlap(pool->pool, all, dst, ib)) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    const size_t smem = 3 * sizeof(uint32_t) * (size_t)((pool->num_slots + 31) / 32);
    static PerDeviceOnce once;
    if (once.run([](int) {
            return cudaFuncSetAttribute(slots_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        3 * KDA_MAX_POOL_SLOTS / 8);
        }) != cudaSuccess)
        return KDA_ERR_LAUNCH;
    return launch_dependent(slots_copy_kernel, pool_grid(pool, n), ST, smem, stream,
                            pool_args(pool, n, src, dst, dev_status)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

KDA_API int kda_slots_zero(const kda_slot_pool* pool, int32_t n, const int32_t* slots, int32_t* dev_status,
                           cudaStream_t stream)
{
    int rc = check_pool(pool);
    if (rc != KDA_OK) return rc;
    if (n < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (n == 0) return KDA_OK;
    if ((rc = check_ptrs({slots})) != KDA_OK) return rc;
    if (overlap(pool->pool, pool_bytes(pool), slots, sizeof(int32_t) * (size_t)n)) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    return launch_dependent(slots_zero_kernel, pool_grid(pool, n), ST, 0, stream,
                            pool_args(pool, n, nullptr, slots, dev_status)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

KDA_API int kda_slots_compact_plan(const kda_slot_pool* pool, const int32_t* live, int32_t* src, int32_t* dst,
                                   int32_t* remap, cudaStream_t stream)
{
    int rc = check_pool(pool);
    if (rc != KDA_OK) return rc;
    if ((rc = check_ptrs({live, src, dst, remap})) != KDA_OK) return rc;
    const size_t b = sizeof(int32_t) * (size_t)pool->num_slots;
    const void* all[4] = {live, src, dst, remap};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(all[i], b, all[j], b)) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    return launch_dependent(compact_plan_kernel, 1, PT, 0, stream, pool->num_slots, live, src, dst, remap) == cudaSuccess
               ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // extern "C"
