// kda_paged_plan.cuh -- how the rows of an attention call are shared out among CTAs, and how the parts of a
// row's tokens are joined.
//
// The rows of a sequence that share a key head (its tokens times the G query heads of the group, token after
// token) are cut into tiles of rows; a tile sees the tokens that any of its rows sees, cut into tiles of keys.  A
// (tile of rows, key head) is a unit; the key tiles of all units form one line (with `unit` places more a unit, for what a unit
// costs besides), and each CTA takes an equal stretch of it, whatever the lengths.  A unit within one stretch
// is written out; one that stretches cut leaves a part in the workspace for each, which join_kernel adds: at most two parts a CTA.
// Only the GPU knows the lengths: every CTA counts the line and finds where its stretch begins by itself (two
// passes over the sequences by all warps, a microsecond or two; a kernel of its own in front took 8 to 18).
#pragma once

#include "kda_paged.h"
#include "kda_ptx.cuh"

namespace kda {
namespace paged {

struct Start {
    long long line;            // places in all
    int seq, row0, head, at;   // first unit of the CTA's stretch, and where in it the stretch begins
};
struct Cut {
    long long line;
    int begin, row0, rows, head, last;  // the unit that begins in a stretch and ends in that of CTA `last`; rows 0: none
};

struct Plan {
    int rows;       // of a tile
    int keys;       // of a tile, a power of two
    int key_shift;
    int ctas;
    int unit;       // places of a unit besides its key tiles
    int part_rows;  // rows kept of a part
    Cut* cut;           // [ctas]
    float2* ml;         // [ctas][2][part_rows]: largest score (in powers of two), sum of the weights;
    float4* o;          // [ctas][2][D / 4][part_rows], not divided.  0: of a unit that began before, 1: of one that goes on
};

inline size_t lay_out(Plan& p, const PagedArgs& a, int rows, int keys, int ctas, int unit)
{
    p.unit = unit;
    p.rows = rows;
    p.keys = keys;
    for (p.key_shift = 0; (1 << p.key_shift) < keys;) ++p.key_shift;
    p.ctas = ctas;
    p.part_rows = (int)std::min<int64_t>(rows, (int64_t)a.T * a.G);
    unsigned char* w = static_cast<unsigned char*>(a.workspace);
    size_t at = 0;
    const auto take = [&](size_t n) {
        unsigned char* x = w ? w + at : nullptr;
        at += (n + 255) / 256 * 256;
        return x;
    };
    p.cut = reinterpret_cast<Cut*>(take(sizeof(Cut) * ctas));
    const size_t part = (size_t)ctas * 2 * p.part_rows;
    p.ml = reinterpret_cast<float2*>(take(part * sizeof(float2)));
    p.o = reinterpret_cast<float4*>(take(part * a.D * sizeof(float)));
    return at;
}

// First place of CTA c's stretch, and the CTA that has place x.
__device__ __forceinline__ long long stretch(long long line, int c, int ctas) { return line * c / ctas; }
__device__ __forceinline__ int owner(long long line, long long x, int ctas) { return (int)(((x + 1) * ctas + line - 1) / line) - 1; }

// Tokens that rows row0 .. row0 + rows - 1 see: [seen, hi), and lo: seen down to the start of a page or of a tile of `keys` in it.
__device__ __forceinline__ void span(const PagedArgs& a, int keys, int pos0, int kv, int row0, int rows, int& lo, int& seen, int& hi)
{
    lo = seen = 0;
    hi = kv;
    if (!a.causal) return;
    const int p0 = pos0 + group_of(a, row0), p1 = pos0 + group_of(a, row0 + rows - 1);
    hi = max(0, min(kv, p1 + 1));
    if (a.window) {
        seen = min(hi, p0 >= a.window ? p0 - a.window + 1 : 0);
        lo = seen & ~(min(keys, 1 << a.page_shift) - 1);
    }
}

// A walk along a stretch, piece of a unit after piece of a unit.
struct Walk {
    int seq, begin, kv;         // sequence, its first row, its tokens in the cache
    int tokens, all;            // its rows, and times G
    int row0, rows, head;       // the unit
    int lo, seen, hi, n;        // its tokens (from lo on; the first that a row sees) and key tiles
    int t0, t1;                 // the piece's key tiles
    bool act;                   // the piece has something to do
    int from;                   // the piece's first place in the unit
    long long left, x;          // places of the stretch from there on, and places before the unit

    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
    __device__ __forceinline__ int pos0() const { return kv - tokens; }
    __device__ __forceinline__ long long end(const Plan& p) const { return x + n + p.unit; }

    // the sequence, or the first behind it, that has rows
    __device__ __forceinline__ void enter(const PagedArgs& a)
    {
        int e, f = 0;
        for (; seq < a.N; ++seq)
            if (paged_seq(a, seq, begin, e, kv, &f)) {
                tokens = e - begin;
                all = tokens * a.G;
                return;
            }
        left = 0;  // lengths that changed under the call
        all = 0;
        kv = begin = tokens = 0;
    }
    __device__ __forceinline__ void unit(const PagedArgs& a, const Plan& p)
    {
        rows = min(p.rows, all - row0);
        span(a, p.keys, pos0(), kv, row0, rows, lo, seen, hi);
        n = (hi - lo + p.keys - 1) >> p.key_shift;
    }
    __device__ __forceinline__ void piece(const Plan& p)
    {
        const int to = (int)min((long long)n + p.unit, from + left);
        t0 = max(from - p.unit, 0);
        t1 = max(to - p.unit, 0);
        act = t1 > t0 || (n == 0 && from == 0);
    }
    bool begun, new_seq, new_unit;
    __device__ __forceinline__ void start(const Plan& p, const Start& s)
    {
        x = stretch(s.line, blockIdx.x, p.ctas);
        left = stretch(s.line, blockIdx.x + 1, p.ctas) - x;
        seq = s.seq;
        row0 = s.row0;
        head = s.head;
        from = s.at;
        x -= from;
        begun = false;
        new_seq = new_unit = true;
    }
    // On to the next piece; false: the stretch is at its end.  (The one place where each step is taken: several roles of a
    // kernel have it each, and their code shares an instruction cache that units of a tile or two run out of.)
    __device__ __forceinline__ bool step(const PagedArgs& a, const Plan& p)
    {
        if (begun) {
            left -= min((long long)n + p.unit, from + left) - from;
            x += n + p.unit;
            from = 0;
            if (++head == a.Hkv) {
                head = 0;
                row0 += p.rows;
                new_unit = true;
                if (row0 >= all) {
                    row0 = 0;
                    ++seq;
                    new_seq = true;
                }
            }
        }
        begun = true;
        if (left <= 0) return false;
        if (new_seq) {
            enter(a);
            new_seq = false;
            if (left <= 0) return false;
        }
        if (new_unit) {
            unit(a, p);
            new_unit = false;
        }
        piece(p);
        return true;
    }
};

// Places of a tile of rows of one key head.
__device__ __forceinline__ int places(const PagedArgs& a, const Plan& p, int pos0, int kv, int row0, int rows)
{
    int lo, seen, hi;
    span(a, p.keys, pos0, kv, row0, rows, lo, seen, hi);
    return ((hi - lo + p.keys - 1) >> p.key_shift) + p.unit;
}

// Where this CTA's stretch begins, by all its WARPS warps (each a run of sequences).  Ends with a barrier.
template <int WARPS> __device__ void find_start(const PagedArgs& a, const Plan& p, Start& out)
{
    __shared__ long long sums[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (int)(((long long)a.N + WARPS - 1) / WARPS);
    const int s0 = (int)min((long long)a.N, (long long)warp * per), s1 = min(a.N, s0 + per);
    int fault = 0;
    // places of the sequences base + lane, over all key heads
    const auto count = [&](int base, int& begin, int& n, int& kv) {
        int end = 0;
        begin = n = kv = 0;
        if (base + lane < s1 && paged_seq(a, base + lane, begin, end, kv, &fault)) n = end - begin;
        const long long all = (long long)n * a.G;
        long long sum = 0;
        const bool few = all <= 4ll * p.rows;
        if (few)
            for (int r = 0; r < all; r += p.rows) sum += places(a, p, kv - n, kv, r, (int)min((long long)p.rows, all - r));
        for (uint32_t left = __ballot_sync(0xffffffffu, !few); left; left &= left - 1) {  // many tiles: by all lanes
            const int l = __ffs(left) - 1, nn = __shfl_sync(0xffffffffu, n, l), k = __shfl_sync(0xffffffffu, kv, l);
            const long long aa = (long long)nn * a.G;
            long long x = 0;
            for (long long r = (long long)lane * p.rows; r < aa; r += 32ll * p.rows) x += places(a, p, k - nn, k, (int)r, (int)min((long long)p.rows, aa - r));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == l) sum = x;
        }
        return sum * a.Hkv;
    };
    const auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    int begin, n, kv;
    long long mine = 0;
    for (int base = s0; base < s1; base += 32) mine += count(base, begin, n, kv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sums[warp] = mine;
    if (blockIdx.x == 0 && fault) flag_status(a.dev_status, fault);
    __syncthreads();
    long long line = 0, before = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sums[w];
        line += sums[w];
    }
    const long long x = stretch(line, blockIdx.x, p.ctas);
    if (threadIdx.x == 0) out.line = line;
    if (x >= before && x < before + mine) {
        for (int base = s0; base < s1; base += 32) {
            const long long c = count(base, begin, n, kv), upto = before + scan(c);
            const uint32_t hit = __ballot_sync(0xffffffffu, x < upto);
            if (!hit) {
                before = __shfl_sync(0xffffffffu, upto, 31);
                continue;
            }
            const int l = __ffs(hit) - 1;
            long long at = x - __shfl_sync(0xffffffffu, upto - c, l);  // within the sequence
            const int nn = __shfl_sync(0xffffffffu, n, l), k = __shfl_sync(0xffffffffu, kv, l);
            const long long all = (long long)nn * a.G;
            for (long long r0 = 0; r0 < all; r0 += 32ll * p.rows) {
                const long long r = r0 + (long long)lane * p.rows;
                const int cost = r < all ? places(a, p, k - nn, k, (int)r, (int)min((long long)p.rows, all - r)) : 0;
                const long long t = scan((long long)cost * a.Hkv);
                const uint32_t in = __ballot_sync(0xffffffffu, at < t);
                if (!in) {
                    at -= __shfl_sync(0xffffffffu, t, 31);
                    continue;
                }
                if (lane == __ffs(in) - 1) {
                    at -= t - (long long)cost * a.Hkv;
                    out.seq = base + l;
                    out.row0 = (int)r;
                    out.head = (int)(at / cost);
                    out.at = (int)(at % cost);
                }
                break;
            }
            break;
        }
    }
    __syncthreads();
}

// The parts of the unit that begins in stretch blockIdx.x and goes on: a CTA 32 rows, a lane a row, a warp four
// channels at a time (as the parts lie), and the rows turned in shared memory.
constexpr int JT = 256;
template <typename IO, int D> __global__ void __launch_bounds__(JT) join_kernel(const PagedArgs a, const Plan p)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    constexpr int AT_ONCE = 32;  // parts whose maxima and sums are held together
    __shared__ float4 turned[32][D / 4 + 1];
    __shared__ float2 held[AT_ONCE][32];
    const int c0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y * 32 + lane;
    const Cut cut = p.cut[c0];
    if (blockIdx.y * 32 >= cut.rows) return;
    // stretches without a place (fewer places than stretches) left nothing
    const auto used = [&](int s) { return stretch(cut.line, c0 + s, p.ctas) < stretch(cut.line, c0 + s + 1, p.ctas); };
    const auto cell = [&](int s) { return (size_t)(c0 + s) * 2 + (s == 0); };
    const int parts = cut.last - c0 + 1;
    const bool in = r < cut.rows;
    constexpr int GROUPS = D / 4, EACH = GROUPS < 8 ? 1 : GROUPS / 8;
    float m = -INFINITY, l = 0.f;
    bool lost = false;
    float4 y[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < parts; s0 += AT_ONCE) {
        const int n = min(AT_ONCE, parts - s0);
        __syncthreads();
        for (int s = warp; s < n; s += JT / 32) held[s][lane] = in && used(s0 + s) ? p.ml[cell(s0 + s) * p.part_rows + r] : make_float2(-INFINITY, 0.f);
        __syncthreads();
        float next = m;
        for (int s = 0; s < n; ++s) next = fmaxf(next, held[s][lane].x);
        const float base = next == -INFINITY ? 0.f : next, f0 = exp2f(m - base);
        m = next;
        l *= f0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) y[i] = make_float4(y[i].x * f0, y[i].y * f0, y[i].z * f0, y[i].w * f0);
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float2 x = held[s][lane];
            lost |= x.y < 0.f;
            if (x.y == 0.f) continue;  // a part that saw nothing, or none (one that met only NaN has no maximum either, but its sum)
            const float f = exp2f(x.x - base);
            l += f * x.y;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const float4 z = p.o[(cell(s0 + s) * GROUPS + warp * EACH + i) * p.part_rows + r];
                y[i].x = fmaf(f, z.x, y[i].x);
                y[i].y = fmaf(f, z.y, y[i].y);
                y[i].z = fmaf(f, z.z, y[i].z);
                y[i].w = fmaf(f, z.w, y[i].w);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        turned[lane][warp * EACH + i] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y[i].x * inv, y[i].y * inv, y[i].z * inv, y[i].w * inv);
    const auto row_of = [&](int rr) {
        const int f = cut.row0 + blockIdx.y * 32 + rr, tok = group_of(a, f);
        return (size_t)(cut.begin + tok) * a.Hq + cut.head * a.G + f - tok * a.G;
    };
    const uint32_t kept = __ballot_sync(0xffffffffu, in && !lost);
    if (a.lse && warp == 0 && ((kept >> lane) & 1)) a.lse[row_of(lane)] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    __syncthreads();
    for (int rr = warp; rr < 32; rr += JT / 32) {
        if (!((kept >> rr) & 1)) continue;
        IO* out = static_cast<IO*>(a.out) + row_of(rr) * D;
        for (int i = lane; i < GROUPS; i += 32) {
            const float4 z = turned[rr][i];
            if constexpr (sizeof(IO) == 4) {
                reinterpret_cast<float4*>(out)[i] = z;
            } else {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(z.x, z.y), hi = __floats2bfloat162_rn(z.z, z.w);
                reinterpret_cast<uint2*>(out)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
        }
    }
}
template <typename IO, int D> cudaError_t launch_join(const PagedArgs& a, const Plan& p, cudaStream_t st)
{
    return launch_dependent(join_kernel<IO, D>, dim3(p.ctas, (p.part_rows + 31) / 32), JT, 0, st, a, p);
}

}  // namespace paged
}  // namespace kda
