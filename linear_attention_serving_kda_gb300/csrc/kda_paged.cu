// kda_paged.cu -- rotary positions, the append of rows to a paged cache, and the
// entry points of the attention over it (kernels: kda_paged_*.cu).
//
// The rotation and the append read and write every value once; HBM bandwidth
// bounds both, and the latency of one pass where rows are few.  A thread holds
// one place of a pair (16 bytes of either half) and goes through the heads with
// it, so that a sine and cosine serve a row's heads.  Measured: rotation of 32768
// rows of 40 heads of 128, bf16, 98 us, 6.8 TB/s (the copy rate); append of 32768
// rows of 48 heads, call after call, 120 us, 6.7 TB/s; 64 rows of single tokens 2.9
// and 4.3 us.
#include <cmath>
#include <cstring>

#include "kda_paged.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

// ------------------------------------------------------------ rotation

// V neighbouring values of a row.
template <typename IO, int V> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
    __device__ __forceinline__ uint32_t* words() { return &r.x; }
};
template <> struct Piece<__nv_bfloat16, 4> {
    uint2 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = r; }
    __device__ __forceinline__ uint32_t* words() { return &r.x; }
};
template <> struct Piece<__nv_bfloat16, 1> {
    __nv_bfloat16 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *p; }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = r; }
};
template <> struct Piece<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = r; }
};
template <> struct Piece<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float* p) { r = *p; }
    __device__ __forceinline__ void store(float* p) const { *p = r; }
};
template <typename IO, int V> __device__ __forceinline__ void widen(Piece<IO, V>& p, float (&x)[V])
{
    if constexpr (sizeof(IO) == 2 && V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const uint32_t w = p.words()[i];
            x[2 * i] = __uint_as_float(w << 16);
            x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
        }
    } else if constexpr (sizeof(IO) == 2) {
        x[0] = __bfloat162float(p.r);
    } else if constexpr (V == 4) {
        x[0] = p.r.x; x[1] = p.r.y; x[2] = p.r.z; x[3] = p.r.w;
    } else {
        x[0] = p.r;
    }
}
template <typename IO, int V> __device__ __forceinline__ void narrow(Piece<IO, V>& p, const float (&x)[V])
{
    if constexpr (sizeof(IO) == 2 && V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            p.words()[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    } else if constexpr (sizeof(IO) == 2) {
        p.r = __float2bfloat16_rn(x[0]);
    } else if constexpr (V == 4) {
        p.r = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        p.r = x[0];
    }
}

struct Turn {
    int rd, pairs_layout;
    float amp, amp_sin;  // amplitude of the cosine and of the sine (negative: the other way)
    const uint64_t* turns;
};

// A unit is V pairs of a head (two pieces of V values), or two pieces behind the rotated channels.  A thread
// keeps a unit of a row over several heads, so that the pairs' sines are formed once for them.
template <typename IO, int V> struct Unit {
    int at, second;   // its pieces' first values within a head
    bool turned;
    float c[V], s[V];
    __device__ __forceinline__ void place(const Turn& t, int u)
    {
        const int p = u * V;
        turned = 2 * p < t.rd;
        at = turned && !t.pairs_layout ? p : 2 * p;
        second = turned && !t.pairs_layout ? p + t.rd / 2 : 2 * p + V;
    }
    // position * turns modulo 2^64 is the angle's part of a turn, exactly; its upper half goes
    // to fp32 (2^-25 of half a turn) and on to sine and cosine of pi times that.
    __device__ __forceinline__ void angles(const Turn& t, int u, int position)
    {
        if (!turned) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t x = __ldg(t.turns + u * V + i) * (uint64_t)(int64_t)position;
            float sn, cs;
            sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &sn, &cs);
            c[i] = t.amp * cs;
            s[i] = t.amp_sin * sn;
        }
    }
    __device__ __forceinline__ void turn(const Turn& t, Piece<IO, V>& p0, Piece<IO, V>& p1) const
    {
        if (!turned) return;
        float x[V], y[V];
        widen(p0, x);
        widen(p1, y);
        if (t.pairs_layout) {
            if constexpr (V == 1) {
                const float a = x[0] * c[0] - y[0] * s[0], b = y[0] * c[0] + x[0] * s[0];
                x[0] = a; y[0] = b;
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1], d = y[2 * i], e = y[2 * i + 1];
                    x[2 * i] = a * c[i] - b * s[i];
                    x[2 * i + 1] = b * c[i] + a * s[i];
                    y[2 * i] = d * c[V / 2 + i] - e * s[V / 2 + i];
                    y[2 * i + 1] = e * c[V / 2 + i] + d * s[V / 2 + i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float a = x[i] * c[i] - y[i] * s[i], b = y[i] * c[i] + x[i] * s[i];
                x[i] = a; y[i] = b;
            }
        }
        narrow(p0, x);
        narrow(p1, y);
    }
};

constexpr int RT = 512;    // most threads of a CTA
// Heads whose loads a thread has in flight together: more take registers from other CTAs (append of 32768 rows of 48 heads of
// 128, a call by itself: 138 us with one, 127 with two, 129 with three, 134 with four, and of single tokens of 64 sequences 4.2, 4.3, 4.5 and
// 3.5 us, of 200 4.3, 4.4, 4.5 and 6.3; rotation of 32768 rows of 40 heads: 105 with one, 99 with two, 98 with four).
constexpr int RAHEAD = 4, AAHEAD = 2;

struct RopeArgs {
    int H, D, units, groups, rows_per_cta;
    long long rows, xs, ys;
    Turn turn;
    const int32_t* positions;
    const void* x;
    void* y;
};

template <typename IO, int V> __global__ void __launch_bounds__(RT) rope_kernel(const RopeArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const IO* xb = static_cast<const IO*>(a.x);
    IO* yb = static_cast<IO*>(a.y);
    for (int i = threadIdx.x; i < a.rows_per_cta * a.groups * a.units; i += blockDim.x) {
        const int u = i % a.units, g = i / a.units % a.groups;
        const long long row = (long long)blockIdx.x * a.rows_per_cta + i / (a.units * a.groups);
        if (row >= a.rows) break;
        const int pos = a.positions[row];
        if (pos < 0) continue;
        Unit<IO, V> w;
        w.place(a.turn, u);
        if (!w.turned && xb == yb) continue;
        const IO* x = xb + row * a.xs;
        IO* y = yb + row * a.ys;
        Piece<IO, V> p[RAHEAD][2];
        auto fetch = [&](int h) {
#pragma unroll
            for (int j = 0; j < RAHEAD; ++j)
                if (h + j * a.groups < a.H) {
                    p[j][0].load(x + (long long)(h + j * a.groups) * a.D + w.at);
                    p[j][1].load(x + (long long)(h + j * a.groups) * a.D + w.second);
                }
        };
        fetch(g);
        w.angles(a.turn, u, pos);
        for (int h = g; h < a.H;) {
#pragma unroll
            for (int j = 0; j < RAHEAD; ++j)
                if (h + j * a.groups < a.H) {
                    w.turn(a.turn, p[j][0], p[j][1]);
                    p[j][0].store(y + (long long)(h + j * a.groups) * a.D + w.at);
                    p[j][1].store(y + (long long)(h + j * a.groups) * a.D + w.second);
                }
            h += RAHEAD * a.groups;
            if (h < a.H) fetch(h);
        }
    }
}

// ------------------------------------------------------------ append

struct AppendArgs {
    PagedArgs p;  // q, k, v: the rows
    int units, groups, rows_per_cta, heads_q;  // heads_q: 0 without queries
    long long qis, ks, vs;
    Turn turn;
    const int32_t* positions;
    void* q_out;
    void* k_cache;
    void* v_cache;
};

constexpr int AROWS = 64;  // most rows of a CTA

// Rows of the CTA first: their sequence (a search), place in the cache and angle, by a thread each.
// Then units as in rope_kernel over the q, k and v heads.
template <typename IO, int V> __global__ void __launch_bounds__(RT) append_kernel(const AppendArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ long long place[AROWS];
    __shared__ int angle[AROWS];
    const PagedArgs& p = a.p;
    const long long row0 = (long long)blockIdx.x * a.rows_per_cta;
    if (blockIdx.x == 0) {  // faults of whole sequences
        int fault = 0, b, e, kv;
        for (int s = threadIdx.x; s < p.N; s += blockDim.x) paged_seq(p, s, b, e, kv, &fault);
        if (fault) flag_status(p.dev_status, fault);
    }
    for (int i = threadIdx.x; i < a.rows_per_cta; i += blockDim.x) {
        long long at = -1;
        const long long row = row0 + i;
        if (row < p.T) {
            int s = (int)row;
            if (p.cu_seqlens) {  // the last sequence that begins at or before the row
                int lo = 0, hi = p.N;
                while (hi - lo > 1) {
                    const int mid = (int)(((unsigned)lo + (unsigned)hi) / 2);
                    if (p.cu_seqlens[mid] <= row) lo = mid;
                    else hi = mid;
                }
                s = lo;
            }
            int begin, end, kv, fault = 0;
            if (paged_seq(p, s, begin, end, kv, &fault) && row >= begin && row < end) {
                fault = 0;
                const long long pos = (long long)kv - (end - row);
                angle[i] = a.positions ? a.positions[row] : (int)pos;
                if (pos < 0) {
                    fault = KDA_DEV_BAD_SEQLENS;
                } else {
                    const int page = p.pages[(long long)s * p.width + (pos >> p.page_shift)];
                    if (page < 0 || page >= p.num_pages) fault = KDA_DEV_BAD_PAGE;
                    else at = page * p.page_stride + (pos & ((1 << p.page_shift) - 1)) * p.token_stride;
                }
                if (fault) flag_status(p.dev_status, fault);
            }
        }
        place[i] = at;
    }
    __syncthreads();
    const int H = a.heads_q + 2 * p.Hkv, D = p.D;
    for (int i = threadIdx.x; i < a.rows_per_cta * a.groups * a.units; i += blockDim.x) {
        const int u = i % a.units, g = i / a.units % a.groups, r = i / (a.units * a.groups);
        const long long row = row0 + r, at = place[r];
        if (at < 0) continue;
        Unit<IO, V> w, flat;  // values are copied piece by piece, as if nothing turned
        w.place(a.turn, u);
        flat.turned = false;
        flat.at = 2 * V * u;
        flat.second = flat.at + V;
        Piece<IO, V> x[AAHEAD][2];
        auto fetch = [&](int h0) {
#pragma unroll
            for (int j = 0; j < AAHEAD; ++j) {
                const int h = h0 + j * a.groups;
                if (h >= H) continue;
                const IO* src = h < a.heads_q           ? static_cast<const IO*>(p.q) + row * a.qis + (long long)h * D
                                : h < a.heads_q + p.Hkv ? static_cast<const IO*>(p.k) + row * a.ks + (long long)(h - a.heads_q) * D
                                                        : static_cast<const IO*>(p.v) + row * a.vs + (long long)(h - a.heads_q - p.Hkv) * D;
                const bool value = h >= a.heads_q + p.Hkv;
                x[j][0].load(src + (value ? flat.at : w.at));
                x[j][1].load(src + (value ? flat.second : w.second));
            }
        };
        fetch(g);
        w.angles(a.turn, u, angle[r]);
        for (int h0 = g; h0 < H;) {
#pragma unroll
            for (int j = 0; j < AAHEAD; ++j) {
                const int h = h0 + j * a.groups;
                if (h >= H) continue;
                const bool value = h >= a.heads_q + p.Hkv;
                IO* dst = h < a.heads_q ? static_cast<IO*>(a.q_out) + row * p.q_stride + (long long)h * D
                          : !value      ? static_cast<IO*>(a.k_cache) + at + (h - a.heads_q) * p.head_stride
                                        : static_cast<IO*>(a.v_cache) + at + (h - a.heads_q - p.Hkv) * p.head_stride;
                if (!value) w.turn(a.turn, x[j][0], x[j][1]);
                x[j][0].store(dst + (value ? flat.at : w.at));
                x[j][1].store(dst + (value ? flat.second : w.second));
            }
            h0 += AAHEAD * a.groups;
            if (h0 < H) fetch(h0);
        }
    }
}

// Values of a piece: 16 bytes where half of the rotated channels is a multiple of that.
int piece_of(int rd, int io_bf16)
{
    if (io_bf16 && rd % 16 == 0) return 8;
    return rd % 8 == 0 ? 4 : 1;
}

// Threads for each row and unit (`groups`), rows of a CTA and its threads: a head a thread until half of the GPU's threads
// are taken, then up to eight heads, which share their angles (2000 rows of 40 heads of 128, the same again and again: 10.4 us where all threads
// are to be taken first, 8.5 so, 7.9 with a quarter; 7001 rows of 12 fp32 heads of 64 7.4, 7.6, 9.0).  CTAs of 128 threads or a row: rotation of
// 32768 rows of 40 heads 99 us with 256, 98 with 128, 115 with 64, of 8192 fp32 rows of 16 heads 20.5, 19.2, 19.1, append of 32768 rows 129, 127, 137.
void split_rows(long long rows, int heads, int units, int max_rows, int& groups, int& rows_per_cta, int& threads)
{
    const long long all = rows * heads * units;
    int per = (int)std::min<long long>(8, std::max<long long>(1, all / (152 * 1024)));
    while ((long long)((heads + per - 1) / per) * units > RT && per < heads) ++per;
    groups = (heads + per - 1) / per;
    rows_per_cta = std::min(std::max(1, 128 / (groups * units)), max_rows);
    threads = std::min(RT, (rows_per_cta * groups * units + 31) / 32 * 32);
}

int check_turn(int D, int rd, int layout, float amp, const uint64_t* turns)
{
    if (rd < 2 || rd > D || rd % 2 != 0) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (layout != KDA_ROPE_HALF && layout != KDA_ROPE_PAIRS) return KDA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(amp)) return KDA_ERR_INVALID_ARGUMENT;
    return check_ptrs({turns});
}

constexpr int64_t MAX_STRIDE = (int64_t)1 << 28;

// A row stride: 0, or at least `dense`, whole 16-byte pieces, within the limit.
bool good_stride(int64_t s, int64_t dense, int64_t unit) { return s == 0 || (s >= dense && s % unit == 0 && s <= MAX_STRIDE); }

int check_paged(const kda_paged_params* p)
{
    if (!p) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_heads_kv <= 0 || p->num_heads_q <= 0 || p->num_heads_q > 1024 || p->num_heads_q % p->num_heads_kv != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    const int D = p->head_dim;
    if (!(D == 32 || D == 64 || D == 128 || D == 256)) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (!known_dtype(p->io_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    const int P = p->page_size;
    if (P < 16 || P > 1024 || (P & (P - 1)) != 0) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (p->num_pages <= 0 || p->pages_per_seq <= 0 || (int64_t)p->pages_per_seq * P > KDA_MAX_ROWS) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t unit = 16 / io_size(p->io_dtype);
    const int64_t ts = p->cache_token_stride ? p->cache_token_stride : (int64_t)p->num_heads_kv * D;
    const int64_t hs = p->cache_head_stride ? p->cache_head_stride : D;
    const int64_t ps = p->cache_page_stride ? p->cache_page_stride : (int64_t)P * p->num_heads_kv * D;
    for (int64_t s : {ts, hs, ps})
        if (s < D || s % unit != 0 || s > ((int64_t)1 << 36)) return KDA_ERR_INVALID_ARGUMENT;
    // places apart: heads within tokens or tokens within heads, and both within a page
    const int64_t heads = (p->num_heads_kv - 1) * hs + D, tokens = (P - 1) * ts + D;
    if (!(p->num_heads_kv == 1 || ts >= heads || hs >= tokens)) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_heads_kv == 1 && ts < D) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_pages > 1 && ps < heads + (P - 1) * ts) return KDA_ERR_INVALID_ARGUMENT;
    if (p->num_pages - 1 > ((int64_t)1 << 60) / ps) return KDA_ERR_INVALID_ARGUMENT;  // (its bytes are counted in 64 bits)
    const int64_t kw = (int64_t)p->num_heads_kv * D, qw = (int64_t)p->num_heads_q * D;
    if (!good_stride(p->q_in_row_stride, qw, unit) || !good_stride(p->q_row_stride, qw, unit) ||
        !good_stride(p->k_row_stride, kw, unit) || !good_stride(p->v_row_stride, kw, unit))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

int check_attn(const kda_paged_params* p)
{
    const int rc = check_paged(p);
    if (rc != KDA_OK) return rc;
    if (!(p->scale > 0.0f && std::isfinite(p->scale * 1.4426950408889634f))) return KDA_ERR_INVALID_ARGUMENT;  // (the kernels count in powers of two)
    if ((p->causal != 0 && p->causal != 1) || p->window < 0 || (p->window > 0 && !p->causal)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

int log2i(int x)
{
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

void fill_paged(PagedArgs& a, const kda_paged_params* p)
{
    std::memset(&a, 0, sizeof(a));
    a.Hq = p->num_heads_q;
    a.Hkv = p->num_heads_kv;
    a.G = a.Hq / a.Hkv;
    const int bits = log2i(a.G);
    a.g_mul = (uint32_t)(((uint64_t)1 << (31 + bits)) / a.G + 1);
    a.g_shift = 31 + bits;
    a.D = p->head_dim;
    a.page_shift = log2i(p->page_size);
    a.num_pages = p->num_pages;
    a.width = p->pages_per_seq;
    a.causal = p->causal;
    a.window = p->window;
    a.scale = p->scale;
    a.token_stride = p->cache_token_stride ? p->cache_token_stride : (int64_t)a.Hkv * a.D;
    a.head_stride = p->cache_head_stride ? p->cache_head_stride : a.D;
    a.page_stride = p->cache_page_stride ? p->cache_page_stride : (int64_t)p->page_size * a.Hkv * a.D;
    a.q_stride = p->q_row_stride ? p->q_row_stride : (int64_t)a.Hq * a.D;
}

size_t cache_bytes(const PagedArgs& a, int io)
{
    const int64_t P = (int64_t)1 << a.page_shift;
    return (size_t)((a.num_pages - 1) * a.page_stride + (P - 1) * a.token_stride + (a.Hkv - 1) * a.head_stride + a.D) * io;
}

size_t strided(int64_t rows, int64_t stride, int64_t width, int io) { return (size_t)((rows - 1) * stride + width) * io; }

// Whether a cache and one of the same strides d elements on share a place.  Pages, and tokens and heads in either order, lie one within the other, so that
// only the two nearest numbers of each stride can bring the places together.
bool places_meet(const PagedArgs& a, int64_t d)
{
    const int64_t P = (int64_t)1 << a.page_shift;
    const bool heads_inside = a.Hkv == 1 || a.token_stride >= (a.Hkv - 1) * a.head_stride + a.D;
    const int64_t stride[3] = {a.num_pages > 1 ? a.page_stride : (int64_t)1 << 60, heads_inside ? a.token_stride : a.head_stride, heads_inside ? a.head_stride : a.token_stride};
    const int64_t count[3] = {a.num_pages, heads_inside ? P : a.Hkv, heads_inside ? a.Hkv : P};
    for (int which = 0; which < 8; ++which) {
        int64_t left = d;
        bool in = true;
        for (int i = 0; i < 3 && in; ++i) {
            int64_t n = left / stride[i];
            if (left < 0 && left % stride[i] != 0) --n;  // down
            n += (which >> i) & 1;
            in = n < count[i] && -n < count[i];
            left -= n * stride[i];
        }
        if (in && left < a.D && -left < a.D) return true;
    }
    return false;
}

template <class F> bool disjoint(const void* const* out, const size_t* nout, int n, const void* const* in, const size_t* nin, int m, F&& same)
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < m; ++j)
            if (overlap(out[i], nout[i], in[j], nin[j]) && !same(i, j)) return false;
    return true;
}

int append(const kda_paged_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens, const int32_t* pages,
           const int32_t* positions, const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
           int32_t* dev_status, cudaStream_t stream)
{
    int rc;
    AppendArgs a = {};
    fill_paged(a.p, p);
    const int io = io_size(p->io_dtype);
    const size_t cache = cache_bytes(a.p, io);
    if (overlap(k_cache, cache, v_cache, cache) && places_meet(a.p, (static_cast<const char*>(v_cache) - static_cast<const char*>(k_cache)) / io))
        return KDA_ERR_INVALID_ARGUMENT;
    if (p->rotary_dim != 0 && (rc = check_turn(p->head_dim, p->rotary_dim, p->rope_layout, p->rope_amplitude, p->rope_turns)) != KDA_OK) return rc;
    if ((rc = check_ptrs({kv_lens, pages, k, v, k_cache, v_cache})) != KDA_OK || (rc = check_opt(positions)) != KDA_OK ||
        (rc = check_opt(q)) != KDA_OK || (rc = check_opt(q_out)) != KDA_OK)
        return rc;
    if ((q == nullptr) != (q_out == nullptr)) return KDA_ERR_INVALID_ARGUMENT;
    a.p.N = N;
    a.p.T = T;
    const int64_t kw = (int64_t)a.p.Hkv * a.p.D, qw = (int64_t)a.p.Hq * a.p.D;
    a.qis = p->q_in_row_stride ? p->q_in_row_stride : qw;
    a.ks = p->k_row_stride ? p->k_row_stride : kw;
    a.vs = p->v_row_stride ? p->v_row_stride : kw;
    const size_t nq = strided(T, a.qis, qw, io), nqo = strided(T, a.p.q_stride, qw, io);
    const void* out[3] = {k_cache, v_cache, q_out};
    const size_t nout[3] = {cache, cache, nqo};
    const void* in[8] = {q, k, v, cu_seqlens, kv_lens, pages, positions, p->rotary_dim ? p->rope_turns : nullptr};
    const size_t nin[8] = {nq, strided(T, a.ks, kw, io), strided(T, a.vs, kw, io), ((size_t)N + 1) * 4, (size_t)N * 4,
                           (size_t)N * p->pages_per_seq * 4, (size_t)T * 4, (size_t)p->rotary_dim * 4};
    const bool in_place = q == q_out && a.qis == a.p.q_stride;
    // k and v within the same strides as q (one row of q|k|v channels) share its range without sharing a value when
    // the rows' widths lie apart: only such an in-place call looks at the channels
    auto apart = [&](int i, int j) {
        if (i != 2) return false;
        if (j == 0) return in_place;
        if (j > 2 || !in_place) return false;
        const int64_t d = (static_cast<const char*>(in[j]) - static_cast<const char*>(q)) / io, s = a.qis, js = j == 1 ? a.ks : a.vs;
        return js == s && d >= qw && d + kw <= s;
    };
    if (!disjoint(out, nout, 3, in, nin, 8, apart)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(q_out, nqo, k_cache, cache) || overlap(q_out, nqo, v_cache, cache)) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    a.p.cu_seqlens = cu_seqlens;
    a.p.kv_lens = kv_lens;
    a.p.pages = pages;
    a.p.q = q; a.p.k = k; a.p.v = v;
    a.p.dev_status = dev_status;
    a.positions = positions;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.heads_q = q ? a.p.Hq : 0;
    a.turn = {p->rotary_dim, p->rope_layout == KDA_ROPE_PAIRS, p->rope_amplitude, p->rope_amplitude, p->rope_turns};
    const int V = piece_of(p->rotary_dim, io == 2);
    a.units = a.p.D / (2 * V);
    int threads;
    split_rows(T, a.heads_q + 2 * a.p.Hkv, a.units, AROWS, a.groups, a.rows_per_cta, threads);
    const unsigned grid = (unsigned)(((int64_t)T + a.rows_per_cta - 1) / a.rows_per_cta);
    const cudaError_t e = io == 4  ? (V == 4 ? launch_dependent(append_kernel<float, 4>, grid, threads, 0, stream, a)
                                             : launch_dependent(append_kernel<float, 1>, grid, threads, 0, stream, a))
                          : V == 8 ? launch_dependent(append_kernel<__nv_bfloat16, 8>, grid, threads, 0, stream, a)
                          : V == 4 ? launch_dependent(append_kernel<__nv_bfloat16, 4>, grid, threads, 0, stream, a)
                                   : launch_dependent(append_kernel<__nv_bfloat16, 1>, grid, threads, 0, stream, a);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

size_t attn_workspace(const kda_paged_params* p, int32_t N, int32_t T, bool token)
{
    PagedArgs a;
    fill_paged(a, p);
    a.N = N;
    a.T = T;
    const bool f32 = p->io_dtype == KDA_DTYPE_F32;
    return token && paged_token_wanted(a, f32) ? paged_token_workspace_bytes(a) : f32 ? paged_f32_workspace_bytes(a) : paged_bf16_workspace_bytes(a);
}

int attend(const kda_paged_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens, const int32_t* pages,
           const void* q, const void* k_cache, const void* v_cache, void* out, float* lse, void* workspace, size_t ws_bytes,
           int32_t* dev_status, bool token, cudaStream_t stream, uint32_t polls = PAGED_POLLS, uint32_t unit_polls = PAGED_POLLS, int stalled = -1)
{
    int rc;
    if ((rc = check_ptrs({kv_lens, pages, q, k_cache, v_cache, out})) != KDA_OK || (rc = check_opt(lse)) != KDA_OK) return rc;
    const int io = io_size(p->io_dtype);
    PagedArgs a;
    fill_paged(a, p);
    a.N = N;
    a.T = T;
    const size_t need = attn_workspace(p, N, T, token), cache = cache_bytes(a, io);
    const int64_t qw = (int64_t)a.Hq * a.D;
    const void* o[3] = {out, lse, workspace};
    const size_t no[3] = {(size_t)T * qw * io, (size_t)T * a.Hq * 4, need};
    const void* in[6] = {q, k_cache, v_cache, cu_seqlens, kv_lens, pages};
    const size_t ni[6] = {strided(T, a.q_stride, qw, io), cache, cache, ((size_t)N + 1) * 4, (size_t)N * 4, (size_t)N * p->pages_per_seq * 4};
    if (!disjoint(o, no, 3, in, ni, 6, [](int, int) { return false; }) || overlap(o[0], no[0], o[1], no[1]) ||
        overlap(o[0], no[0], o[2], no[2]) || overlap(o[1], no[1], o[2], no[2]))
        return KDA_ERR_INVALID_ARGUMENT;
    if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return KDA_ERR_WORKSPACE;
    if ((rc = check_device()) != KDA_OK) return rc;
    a.cu_seqlens = cu_seqlens;
    a.kv_lens = kv_lens;
    a.pages = pages;
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.dev_status = dev_status;
    a.polls = polls;
    a.unit_polls = unit_polls;
    a.stalled = stalled;
    const cudaError_t e = token && paged_token_wanted(a, io == 4) ? launch_paged_token(a, io == 4, stream)
                          : io == 4                               ? launch_paged_f32(a, stream)
                                                                  : launch_paged_bf16(a, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

// Sequences and rows of a call within the index range (row tiles and heads of all of them are counted in 32 bits).
bool good_counts(const kda_paged_params* p, int64_t N, int64_t T)
{
    return N >= 0 && T >= 0 && N <= KDA_MAX_ROWS - 1024 && T <= KDA_MAX_ROWS && (T + N) * p->num_heads_q <= INT32_MAX - 65536;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

KDA_API int kda_rope_turns(const kda_rope_scaling* s, int32_t rotary_dim, const double* radians, uint64_t* turns)
{
    if (!s || !turns) return KDA_ERR_INVALID_ARGUMENT;
    if (rotary_dim < 2 || rotary_dim > KDA_ROPE_MAX_DIM || rotary_dim % 2 != 0) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    const int kind = s->kind, n = rotary_dim / 2;
    const double two_pi = 6.283185307179586476925286766559;
    if (kind < KDA_ROPE_SCALE_NONE || kind > KDA_ROPE_SCALE_SMOOTH) return KDA_ERR_INVALID_ARGUMENT;
    if (!(radians && kind != KDA_ROPE_SCALE_RAMP) && !(std::isfinite(s->base) && s->base > 1.0)) return KDA_ERR_INVALID_ARGUMENT;
    if (kind != KDA_ROPE_SCALE_NONE && !(std::isfinite(s->factor) && s->factor > 0.0)) return KDA_ERR_INVALID_ARGUMENT;
    if (kind == KDA_ROPE_SCALE_BASE && (radians || rotary_dim == 2)) return KDA_ERR_INVALID_ARGUMENT;
    if (kind == KDA_ROPE_SCALE_RAMP || kind == KDA_ROPE_SCALE_SMOOTH)
        if (!(std::isfinite(s->length) && s->length > 0.0 && std::isfinite(s->fast) && s->slow > 0.0 && s->fast > s->slow))
            return KDA_ERR_INVALID_ARGUMENT;
    if (radians)
        for (int i = 0; i < n; ++i)
            if (!std::isfinite(radians[i])) return KDA_ERR_INVALID_ARGUMENT;
    const double base = kind == KDA_ROPE_SCALE_BASE ? s->base * std::pow(s->factor, (double)rotary_dim / (rotary_dim - 2)) : s->base;
    if (kind == KDA_ROPE_SCALE_BASE && !(std::isfinite(base) && base > 0.0)) return KDA_ERR_INVALID_ARGUMENT;
    double low = 0, high = 1;
    if (kind == KDA_ROPE_SCALE_RAMP) {
        const auto dim = [&](double b) { return rotary_dim * std::log(s->length / (b * two_pi)) / (2 * std::log(s->base)); };
        low = std::max(std::floor(dim(s->fast)), 0.0);
        high = std::min(std::ceil(dim(s->slow)), rotary_dim - 1.0);
    }
    for (int i = 0; i < n; ++i) {
        double f = radians ? radians[i] : std::pow(base, -2.0 * i / rotary_dim);
        if (kind == KDA_ROPE_SCALE_LINEAR) f /= s->factor;
        if (kind == KDA_ROPE_SCALE_RAMP) {
            const double r = std::min(std::max((i - low) / std::max(high - low, 1e-3), 0.0), 1.0);
            f = f * (1 - r) + f / s->factor * r;
        }
        if (kind == KDA_ROPE_SCALE_SMOOTH) {
            const double k = std::min(std::max((s->length * f / two_pi - s->slow) / (s->fast - s->slow), 0.0), 1.0);
            f = f * k + f / s->factor * (1 - k);
        }
        if (!std::isfinite(f)) return KDA_ERR_INVALID_ARGUMENT;
        double t = f / two_pi;
        t -= std::floor(t);
        turns[i] = t >= 1.0 ? 0 : (uint64_t)std::ldexp(t, 64);
    }
    return KDA_OK;
}

KDA_API int kda_rope(const kda_rope_params* p, int64_t rows, const int32_t* positions, const void* x, void* y, cudaStream_t stream)
{
    if (!p || p->num_heads <= 0 || !known_dtype(p->io_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (p->head_dim < 16 || p->head_dim > KDA_ROPE_MAX_DIM || p->head_dim % 16 != 0) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    int rc = check_turn(p->head_dim, p->rotary_dim, p->rope_layout, p->rope_amplitude, p->rope_turns);
    if (rc != KDA_OK) return rc;
    if (p->transpose != 0 && p->transpose != 1) return KDA_ERR_INVALID_ARGUMENT;
    const int io = io_size(p->io_dtype);
    const int64_t dense = (int64_t)p->num_heads * p->head_dim;
    if (dense > MAX_STRIDE || !good_stride(p->x_row_stride, dense, 16 / io) || !good_stride(p->y_row_stride, dense, 16 / io)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows < 0 || rows > KDA_MAX_ROWS) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0) return KDA_OK;
    if ((rc = check_ptrs({positions, x, y})) != KDA_OK) return rc;
    RopeArgs a;
    a.xs = p->x_row_stride ? p->x_row_stride : dense;
    a.ys = p->y_row_stride ? p->y_row_stride : dense;
    const size_t ny = strided(rows, a.ys, dense, io);
    if (!(x == y && a.xs == a.ys) && overlap(x, strided(rows, a.xs, dense, io), y, ny)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(y, ny, positions, (size_t)rows * 4) || overlap(y, ny, p->rope_turns, (size_t)p->rotary_dim * 4)) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    a.H = p->num_heads;
    a.D = p->head_dim;
    a.rows = rows;
    a.turn = {p->rotary_dim, p->rope_layout == KDA_ROPE_PAIRS, p->rope_amplitude, p->transpose ? -p->rope_amplitude : p->rope_amplitude, p->rope_turns};
    a.positions = positions;
    a.x = x;
    a.y = y;
    const int V = piece_of(p->rotary_dim, io == 2);
    a.units = a.D / (2 * V);
    int threads;
    split_rows(rows, a.H, a.units, 1 << 20, a.groups, a.rows_per_cta, threads);
    const unsigned grid = (unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta);
    const cudaError_t e = io == 4  ? (V == 4 ? launch_dependent(rope_kernel<float, 4>, grid, threads, 0, stream, a)
                                             : launch_dependent(rope_kernel<float, 1>, grid, threads, 0, stream, a))
                          : V == 8 ? launch_dependent(rope_kernel<__nv_bfloat16, 8>, grid, threads, 0, stream, a)
                          : V == 4 ? launch_dependent(rope_kernel<__nv_bfloat16, 4>, grid, threads, 0, stream, a)
                                   : launch_dependent(rope_kernel<__nv_bfloat16, 1>, grid, threads, 0, stream, a);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

KDA_API int kda_paged_append_varlen(const kda_paged_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens,
                                    const int32_t* pages, const int32_t* positions, const void* q, const void* k, const void* v,
                                    void* q_out, void* k_cache, void* v_cache, int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_paged(p);
    if (rc != KDA_OK) return rc;
    if (!good_counts(p, N, T)) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0 || T == 0) return KDA_OK;
    if ((rc = check_ptrs({cu_seqlens})) != KDA_OK) return rc;
    return append(p, cu_seqlens, N, T, kv_lens, pages, positions, q, k, v, q_out, k_cache, v_cache, dev_status, stream);
}

KDA_API int kda_paged_append_decode(const kda_paged_params* p, int32_t B, const int32_t* kv_lens, const int32_t* pages, const int32_t* positions,
                                    const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                                    int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_paged(p);
    if (rc != KDA_OK) return rc;
    if (!good_counts(p, B, B)) return KDA_ERR_INVALID_ARGUMENT;
    if (B == 0) return KDA_OK;
    return append(p, nullptr, B, B, kv_lens, pages, positions, q, k, v, q_out, k_cache, v_cache, dev_status, stream);
}

KDA_API size_t kda_paged_attn_workspace_bytes(const kda_paged_params* p, int32_t N, int32_t T)
{
    if (check_attn(p) != KDA_OK || !good_counts(p, N, T) || N == 0 || T == 0) return 0;
    return attn_workspace(p, N, T, false);
}

KDA_API int kda_paged_attn_varlen(const kda_paged_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens,
                                  const int32_t* pages, const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                                  void* workspace, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_attn(p);
    if (rc != KDA_OK) return rc;
    if (!good_counts(p, N, T)) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0 || T == 0) return KDA_OK;
    if ((rc = check_ptrs({cu_seqlens})) != KDA_OK) return rc;
    return attend(p, cu_seqlens, N, T, kv_lens, pages, q, k_cache, v_cache, out, lse, workspace, ws_bytes, dev_status, false, stream);
}

KDA_API size_t kda_paged_attn_decode_workspace_bytes(const kda_paged_params* p, int32_t B)
{
    if (check_attn(p) != KDA_OK || !good_counts(p, B, B) || B == 0) return 0;
    return attn_workspace(p, B, B, true);
}

KDA_API int kda_paged_attn_decode(const kda_paged_params* p, int32_t B, const int32_t* kv_lens, const int32_t* pages, const void* q,
                                  const void* k_cache, const void* v_cache, void* out, float* lse, void* workspace, size_t ws_bytes,
                                  int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_attn(p);
    if (rc != KDA_OK) return rc;
    if (!good_counts(p, B, B)) return KDA_ERR_INVALID_ARGUMENT;
    if (B == 0) return KDA_OK;
    return attend(p, nullptr, B, B, kv_lens, pages, q, k_cache, v_cache, out, lse, workspace, ws_bytes, dev_status, true, stream);
}

KDA_API int kda_debug_paged_attn_stalled(const kda_paged_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens,
                                         const int32_t* pages, const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                                         void* workspace, size_t ws_bytes, int32_t* dev_status, uint32_t poll_limit, uint32_t unit_poll_limit,
                                         int32_t stalled_cta, cudaStream_t stream)
{
    int rc = check_attn(p);
    if (rc != KDA_OK) return rc;
    const bool token = cu_seqlens == nullptr;
    if (!good_counts(p, N, T) || (token && N != T) || poll_limit == 0 || unit_poll_limit == 0) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0 || T == 0) return KDA_OK;
    if (!token && (rc = check_ptrs({cu_seqlens})) != KDA_OK) return rc;
    return attend(p, cu_seqlens, N, T, kv_lens, pages, q, k_cache, v_cache, out, lse, workspace, ws_bytes, dev_status, token, stream, poll_limit,
                  unit_poll_limit, stalled_cta);
}

}  // extern "C"
