// kda_paged_plan.cuh -- how the rows of an attention call are cut into work, and
// how the parts of a long row's tokens are joined.
//
// The rows of a sequence that share a key head (its tokens times the G query heads of the
// group, token after token) are cut into tiles; a tile's tokens are those that any of its rows
// sees.  One CTA takes all of a tile's tokens where there are tiles enough; few rows over many tokens are
// cut along the tokens as well, into items of about half a CTA's share of the whole, and
// joined afterwards.  Only the GPU knows the lengths, so a kernel of one CTA writes the items, longest first.
#pragma once

#include "kda_paged.h"
#include "kda_ptx.cuh"

namespace kda {
namespace paged {

struct Item {
    int begin, seq;         // first row of the sequence; its number
    int row0, rows;         // rows of the tile, counted over tokens and heads of the group
    int pos0;               // token of the sequence's first row
    int k0, k1;             // tokens of this item; k0 starts a page or a tile of one
    int part;               // -1: the whole tile, else where its sums go
};
struct Joined {
    int begin, row0, rows, part, parts;
};
struct Head {
    int items, joined, parts, pad;
};

struct Plan {
    int rows;      // of a tile
    int keys;      // of a tile
    int ctas;      // that share the work
    int max_items, max_joined, max_parts;
    int part_rows; // rows kept of a part
    Head* head;
    Item* items;
    Joined* joined;
    float* o;      // [parts][Hkv][part_rows][D], not divided by the weights' sum
    float2* ml;    // [parts][Hkv][part_rows]: largest score (in powers of two), sum of the weights
};

constexpr int LEAST = 2;  // key tiles of an item, at least

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Bounds and places in the workspace.  A tile cut into parts has more than one item's length L of key
// tiles, so it has at most 2 cost / L parts, and L >= total / (2 ctas): 4 ctas parts over all key heads.
inline size_t lay_out(Plan& p, const PagedArgs& a, int rows, int keys, int ctas)
{
    p.rows = rows;
    p.keys = keys;
    p.ctas = ctas;
    const int64_t tiles = ((int64_t)a.T * a.G + rows - 1) / rows + std::min(a.N, a.T);
    p.max_parts = 4 * ctas / a.Hkv + 2;
    p.max_joined = p.max_parts / 2 + 1;
    p.max_items = (int)(tiles + p.max_parts);
    p.part_rows = (int)std::min<int64_t>(rows, (int64_t)a.T * a.G);
    unsigned char* w = static_cast<unsigned char*>(a.workspace);
    size_t at = 0;
    const auto take = [&](size_t n) {
        unsigned char* x = w ? w + at : nullptr;
        at += align256(n);
        return x;
    };
    p.head = reinterpret_cast<Head*>(take(sizeof(Head)));
    p.items = reinterpret_cast<Item*>(take(sizeof(Item) * (size_t)p.max_items));
    p.joined = reinterpret_cast<Joined*>(take(sizeof(Joined) * (size_t)p.max_joined));
    const size_t part = (size_t)p.max_parts * a.Hkv * p.part_rows;
    p.ml = reinterpret_cast<float2*>(take(part * sizeof(float2)));
    p.o = reinterpret_cast<float*>(take(part * a.D * sizeof(float)));
    return at;
}

// Tokens that rows row0 .. row0 + rows - 1 see: [lo, hi), lo down to the start of a page or of a tile of `keys` in it.
__device__ __forceinline__ void span(const PagedArgs& a, int keys, int pos0, int kv, int row0, int rows, int& lo, int& hi)
{
    lo = 0;
    hi = kv;
    if (!a.causal) return;
    const long long p0 = (long long)pos0 + row0 / a.G, p1 = (long long)pos0 + (row0 + rows - 1) / a.G;
    hi = (int)max(0ll, min((long long)kv, p1 + 1));
    if (a.window) {
        const int unit = min(keys, 1 << a.page_shift);
        lo = (int)min((long long)hi, max(0ll, p0 - a.window + 1)) & ~(unit - 1);
    }
}

constexpr int PT = 1024;
constexpr int BUCKETS = 512;

// f(begin, seq, row0, rows, pos0, lo, hi) for every tile, by one thread each.  Few sequences: the CTA takes the tiles
// of one after the other; many: a warp each.
template <class F> __device__ void each_tile(const PagedArgs& a, const Plan& p, int* fault, F&& f)
{
    const int lane = threadIdx.x & 31;
    const bool wide = a.N <= 16;
    const int team = wide ? PT : 32, who = wide ? threadIdx.x : lane, step = wide ? 1 : PT / 32;
    // sequences first .. first + 31 * step are looked up at a time, one by each lane
    for (long long first = wide ? 0 : threadIdx.x >> 5; first < a.N; first += 32 * step) {
        int begin = 0, end = 0, kv = 0, ok = 0;
        const long long mine = first + (long long)lane * step;
        if (mine < a.N) ok = paged_seq(a, (int)mine, begin, end, kv, fault);
        uint32_t left = __ballot_sync(0xffffffffu, ok);
        while (left) {
            const int l = __ffs(left) - 1;
            left &= left - 1;
            const int b = __shfl_sync(0xffffffffu, begin, l), n = __shfl_sync(0xffffffffu, end, l) - b, t = __shfl_sync(0xffffffffu, kv, l);
            const int all = n * a.G;
            for (long long r = (long long)who * p.rows; r < all; r += (long long)team * p.rows) {
                const int rows = min(p.rows, all - (int)r);
                int lo, hi;
                span(a, p.keys, t - n, t, (int)r, rows, lo, hi);
                f(b, (int)(first + (long long)l * step), (int)r, rows, t - n, lo, hi);
            }
        }
    }
}

static __global__ void __launch_bounds__(PT) plan_kernel(const PagedArgs a, const Plan p)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ unsigned long long total;
    __shared__ int longest, bucket[BUCKETS], njoined, nparts, sums[PT / 32], all_faults;
    const int tid = threadIdx.x;
    if (tid == 0) {
        total = 0;
        longest = njoined = nparts = all_faults = 0;
    }
    for (int i = tid; i < BUCKETS; i += PT) bucket[i] = 0;
    __syncthreads();
    const auto cost = [&](int lo, int hi) { return max(1, (hi - lo + p.keys - 1) / p.keys); };
    {
        long long sum = 0;
        int most = 0, fault = 0;
        each_tile(a, p, &fault, [&](int, int, int, int, int, int lo, int hi) {
            const int c = cost(lo, hi);
            sum += c;
            most = max(most, c);
        });
        if (fault) atomicOr(&all_faults, fault);
        if (sum) {
            atomicAdd(&total, (unsigned long long)sum);
            atomicMax(&longest, most);
        }
    }
    __syncthreads();
    if (tid == 0 && all_faults) flag_status(a.dev_status, all_faults);
    const unsigned long long share = total * a.Hkv / (2u * p.ctas) + 1;
    const int L = (int)min((unsigned long long)INT32_MAX, max((unsigned long long)LEAST, share));
    const int top = min(L, longest);
    const auto bucket_of = [&](int c) { return (int)((long long)(top - min(c, top)) * (BUCKETS - 1) / max(top, 1)); };
    int dummy = 0;
    each_tile(a, p, &dummy, [&](int, int, int, int, int, int lo, int hi) {
        const int c = cost(lo, hi), parts = (c + L - 1) / L;
        atomicAdd(&bucket[bucket_of((c + parts - 1) / parts)], parts);
    });
    __syncthreads();
    // where each bucket begins
    int mine = tid < BUCKETS ? bucket[tid] : 0, before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if ((tid & 31) >= o) before += x;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = before;
    __syncthreads();
    int below = (tid & 31) < (tid >> 5) ? sums[tid & 31] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
    before += below;
    if (tid == BUCKETS - 1) p.head->items = before;
    if (tid < BUCKETS) bucket[tid] = before - mine;
    __syncthreads();
    each_tile(a, p, &dummy, [&](int begin, int seq, int row0, int rows, int pos0, int lo, int hi) {
        const int c = cost(lo, hi), parts = (c + L - 1) / L, each = (c + parts - 1) / parts;
        const int at = atomicAdd(&bucket[bucket_of(each)], parts);
        int part = -1;
        if (parts > 1) {
            part = atomicAdd(&nparts, parts);
            p.joined[atomicAdd(&njoined, 1)] = {begin, row0, rows, part, parts};
        }
        for (int i = 0; i < parts; ++i) {
            // part i's key tiles: c * i / parts and on, none of them empty
            const int t0 = (int)((long long)c * i / parts), t1 = (int)((long long)c * (i + 1) / parts);
            Item it;
            it.begin = begin; it.seq = seq; it.row0 = row0; it.rows = rows; it.pos0 = pos0;
            it.k0 = lo + t0 * p.keys;
            it.k1 = min(hi, lo + t1 * p.keys);
            it.part = parts > 1 ? part + i : -1;
            p.items[at + i] = it;
        }
    });
    __syncthreads();
    if (tid == 0) {
        p.head->joined = njoined;
        p.head->parts = nparts;
    }
}

// A warp joins the parts of one row: part s has its maximum and sum at ml(s) and its D values at o(s), both
// null for a part without any.  Returns the sum and the maximum, and in y the lane's D / 32 neighbouring values, not divided.
template <int D, class ML, class O> __device__ __forceinline__ float2 join_row(int parts, ML&& ml, O&& o, float (&y)[D / 32])
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < parts; s += 32)
        if (const float2* x = ml(s)) m = fmaxf(m, x->x);
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
#pragma unroll 4
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
    return make_float2(m, warp_sum(l));
}
// The joined row to out and lse (row: of [T][Hq]).
template <typename IO, int D> __device__ __forceinline__ void write_row(const PagedArgs& a, size_t row, float2 ml, const float (&y)[D / 32])
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
    IO* out = static_cast<IO*>(a.out) + row * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) stv(out + e, ml.y == 0.f ? 0.f : y[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.69314718055994531f;
}

// Rows whose tokens were cut into parts: a warp a row.
constexpr int JT = 256;
template <typename IO, int D> __global__ void __launch_bounds__(JT) join_kernel(const PagedArgs a, const Plan p)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int rows = p.head->joined * a.Hkv * p.part_rows;
    for (int i = blockIdx.x * (JT / 32) + (threadIdx.x >> 5); i < rows; i += gridDim.x * (JT / 32)) {
        const int r = i % p.part_rows, th = i / p.part_rows, h = th % a.Hkv;
        const Joined j = p.joined[th / a.Hkv];
        if (r >= j.rows) continue;
        const size_t first = ((size_t)j.part * a.Hkv + h) * p.part_rows + r, step = (size_t)a.Hkv * p.part_rows;
        float y[D / 32];
        const float2 ml = join_row<D>(j.parts, [&](int s) { return p.ml + first + s * step; }, [&](int s) { return p.o + (first + s * step) * D; }, y);
        const int f = j.row0 + r;
        write_row<IO, D>(a, (size_t)(j.begin + f / a.G) * a.Hq + h * a.G + f % a.G, ml, y);
    }
}
template <typename IO, int D> cudaError_t launch_join(const PagedArgs& a, const Plan& p, cudaStream_t st)
{
    const int64_t most = ((int64_t)p.max_joined * a.Hkv * p.part_rows + JT / 32 - 1) / (JT / 32);
    return launch_dependent(join_kernel<IO, D>, (unsigned)std::min<int64_t>(most, 152 * 8), JT, 0, st, a, p);
}

}  // namespace paged
}  // namespace kda
