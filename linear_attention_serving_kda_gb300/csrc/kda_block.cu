// kda_block.cu -- the memory-bound operators around a recurrent layer: the
// causal depthwise convolution with carried state and SiLU, and the norms
// around a block.  Each reads and writes every value once; HBM bandwidth
// bounds both.
#include <cmath>

#include "kda_check.h"
#include "kda_common.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace {

// ------------------------------------------------------------ eight values

template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const void* p) { r = *static_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p)
    {
        a = static_cast<const float4*>(p)[0];
        b = static_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(void* p) const
    {
        static_cast<float4*>(p)[0] = a;
        static_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[8])
    {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// ------------------------------------------------------------ convolution

struct ConvArgs {
    int C, N, T, num_slots;
    const int32_t* cu_seqlens;
    const void* x;
    const float* w;
    const int32_t* slots;
    void* state;
    void* y;
    int32_t* dev_status;
};

// Each thread owns eight channels: their K taps in registers, two channels to
// a packed value (fp32 arithmetic of two values an instruction: with single ones the issue
// slots were the bound, 280 us where these take 178), and the last K-1 rows beside them, so a
// tile of rows is read once.  Bound: HBM; 32768 rows of 8192 bf16 channels 176 us, 6.1 TB/s.
template <typename IO, int K> struct ConvLane {
    float2 w[K][4];
    float2 win[K][4];  // win[K-1]: the current row, the ones before it below
    __device__ __forceinline__ void taps(const float* p, int c)
    {
        float f[8 * K];
#pragma unroll
        for (int i = 0; i < 2 * K; ++i) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p + (size_t)c * K) + i);
            f[4 * i] = x.x; f[4 * i + 1] = x.y; f[4 * i + 2] = x.z; f[4 * i + 3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j][i] = make_float2(f[2 * i * K + j], f[(2 * i + 1) * K + j]);
    }
    __device__ __forceinline__ void put(int j, const Vec8<IO>& v)
    {
        float x[8];
        v.get(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) win[j][i] = make_float2(x[2 * i], x[2 * i + 1]);
    }
    // the outputs of the row in win[K-1]; then the window moves on
    __device__ __forceinline__ void step(Vec8<IO>& out)
    {
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 acc = mul2(w[0][i], win[0][i]);
#pragma unroll
            for (int j = 1; j < K; ++j) acc = fma2(w[j][i], win[j][i], acc);
            // x / (1 + e^-x)
            const float2 e = mul2(acc, both2(-1.44269504088896341f));
            const float2 d = add2(make_float2(exp2_sfu(e.x), exp2_sfu(e.y)), both2(1.f));
            const float2 s = mul2(acc, make_float2(rcp_sfu(d.x), rcp_sfu(d.y)));
            y[2 * i] = s.x;
            y[2 * i + 1] = s.y;
        }
        out.set(y);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) win[j][i] = win[j + 1][i];
    }
};

constexpr int CT = 64;        // threads: 512 channels (more, smaller CTAs hide more of the loads: 128 threads took 218 us where these take 178)
constexpr int CONV_AHEAD = 8; // rows loaded at a time, a batch ahead of the one worked on

// Tiles start at a sequence's first row, so only its tile 0 reads the old
// state: that CTA also writes the new one, after its reads, and no other CTA
// touches the slot.  blockIdx.x counts tiles over the sequences.  Six CTAs an SM: five
// (174 registers) took 199 us where these take 178, though four bf16 taps spill 48 bytes of loads for it.
template <typename IO, int K, int CONV_ROWS> __global__ void __launch_bounds__(CT, sizeof(IO) == 2 ? 6 : 1) conv_varlen_kernel(const ConvArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x;
    if ((int)blockIdx.x < a.N && blockIdx.y == 0 && tid == 0) {  // as many CTAs as sequences, at least
        const int f = a.cu_seqlens[blockIdx.x], l = a.cu_seqlens[blockIdx.x + 1];
        if (f < 0 || l < f || l > a.T) flag_status(a.dev_status, KDA_DEV_BAD_SEQLENS);
    }
    int b, e;
    const int seq = find_tile<CONV_ROWS>(a.cu_seqlens, a.N, a.T, blockIdx.x, tid & 31, b, e);
    if (seq < 0) return;
    const int slot = a.slots ? a.slots[seq] : seq;
    if (slot >= a.num_slots) {
        if (tid == 0) flag_status(a.dev_status, KDA_DEV_BAD_SLOT);
        return;
    }
    const int c = (blockIdx.y * CT + tid) * 8;
    if (slot < 0 || c >= a.C) return;
    const int r0 = b + ((int)blockIdx.x - b / CONV_ROWS - seq) * CONV_ROWS, r1 = min(r0 + CONV_ROWS, e);
    const size_t C = a.C;
    const IO* x = static_cast<const IO*>(a.x);
    IO* y = static_cast<IO*>(a.y);
    IO* st = static_cast<IO*>(a.state) + (size_t)slot * (K - 1) * C;

    Vec8<IO> hist[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        hist[j].load(r0 == b ? st + j * C + c : x + (size_t)(r0 - (K - 1) + j) * C + c);
    ConvLane<IO, K> ln;
    ln.taps(a.w, c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) ln.put(j, hist[j]);
    if (r0 == b) {
        // the new state: the last K-1 rows of old state and sequence
        const int len = e - b;
        Vec8<IO> nw[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int r = len - (K - 1) + j;  // row of the sequence; negative: old row K-1+r
            if (r >= 0) nw[j].load(x + (size_t)(b + r) * C + c);
            else {
#pragma unroll
                for (int i = 0; i < K - 1; ++i)
                    if (i == K - 1 + r) nw[j] = hist[i];
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) nw[j].store(st + j * C + c);
    }
    const IO* xp = x + (size_t)r0 * C + c;
    IO* yp = y + (size_t)r0 * C + c;
    int left = r1 - r0;
    Vec8<IO> next[CONV_AHEAD];
    if (left >= CONV_AHEAD)
#pragma unroll
        for (int i = 0; i < CONV_AHEAD; ++i) next[i].load(xp + i * C);
#pragma unroll 1
    for (; left >= CONV_AHEAD; left -= CONV_AHEAD, yp += CONV_AHEAD * C) {
        Vec8<IO> in[CONV_AHEAD];
#pragma unroll
        for (int i = 0; i < CONV_AHEAD; ++i) in[i] = next[i];
        xp += CONV_AHEAD * C;
        if (left >= 2 * CONV_AHEAD)
#pragma unroll
            for (int i = 0; i < CONV_AHEAD; ++i) next[i].load(xp + i * C);
#pragma unroll
        for (int i = 0; i < CONV_AHEAD; ++i) {
            ln.put(K - 1, in[i]);
            Vec8<IO> o;
            ln.step(o);
            o.store(yp + i * C);
        }
    }
#pragma unroll 1
    for (; left > 0; --left, xp += C, yp += C) {
        Vec8<IO> in, o;
        in.load(xp);
        ln.put(K - 1, in);
        ln.step(o);
        o.store(yp);
    }
}

// One row per sequence; a thread takes SEQS of them, so the taps (four bytes a
// weight, as much as the rows) are read once for all: 64 sequences of 8192 bf16
// channels 3.6 us, 7.5 with one each; four of them 3.1 and 3.8.  Bound: latency
// at this size (8.4 MB move in 1.2 us).
constexpr int SEQS = 4;
template <typename IO, int K> __global__ void __launch_bounds__(CT) conv_decode_kernel(const ConvArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int c = (blockIdx.y * CT + threadIdx.x) * 8;
    if (c >= a.C) return;
    const size_t C = a.C;
    int slot[SEQS];
#pragma unroll
    for (int q = 0; q < SEQS; ++q) {
        const int seq = blockIdx.x * SEQS + q;
        slot[q] = seq >= a.N ? -1 : a.slots ? a.slots[seq] : seq;
        if (slot[q] >= a.num_slots) {
            if (threadIdx.x == 0) flag_status(a.dev_status, KDA_DEV_BAD_SLOT);
            slot[q] = -1;
        }
    }
    ConvLane<IO, K> ln;
    Vec8<IO> v[SEQS][K];
#pragma unroll
    for (int q = 0; q < SEQS; ++q)
        if (slot[q] >= 0) {
            const IO* st = static_cast<const IO*>(a.state) + (size_t)slot[q] * (K - 1) * C + c;
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v[q][j].load(st + j * C);
            v[q][K - 1].load(static_cast<const IO*>(a.x) + (size_t)(blockIdx.x * SEQS + q) * C + c);
        }
    ln.taps(a.w, c);
#pragma unroll
    for (int q = 0; q < SEQS; ++q)
        if (slot[q] >= 0) {
#pragma unroll
            for (int j = 0; j < K; ++j) ln.put(j, v[q][j]);
            Vec8<IO> o;
            ln.step(o);
            o.store(static_cast<IO*>(a.y) + (size_t)(blockIdx.x * SEQS + q) * C + c);
            IO* st = static_cast<IO*>(a.state) + (size_t)slot[q] * (K - 1) * C + c;
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v[q][j + 1].store(st + j * C);
        }
}

template <typename IO, int K> cudaError_t launch_conv_decode(const ConvArgs& a, int cols, cudaStream_t st)
{
    return launch_dependent(conv_decode_kernel<IO, K>, dim3((a.N + SEQS - 1) / SEQS, cols), CT, 0, st, a);
}

template <typename IO, int K> cudaError_t launch_conv_varlen(const ConvArgs& a, int cols, cudaStream_t st)
{
    // long tiles (the K-1 rows before a tile and the taps are read again for each) where they
    // still give every SM eight CTAs: 32768 rows of 8192 channels 176 us, 218 with short ones;
    // 333 rows 7.9 us with short ones, 21 with long ones.  Nothing between the two lengths was tried
    if ((long long)(a.T / 128) * cols >= 8LL * sm_count())
        return launch_dependent(conv_varlen_kernel<IO, K, 128>, dim3(a.N + a.T / 128, cols), CT, 0, st, a);
    return launch_dependent(conv_varlen_kernel<IO, K, 16>, dim3(a.N + a.T / 16, cols), CT, 0, st, a);
}

template <typename IO> cudaError_t launch_conv(const ConvArgs& a, int K, bool varlen, cudaStream_t st)
{
    const int cols = (a.C / 8 + CT - 1) / CT;
    if (K == 2) return varlen ? launch_conv_varlen<IO, 2>(a, cols, st) : launch_conv_decode<IO, 2>(a, cols, st);
    if (K == 3) return varlen ? launch_conv_varlen<IO, 3>(a, cols, st) : launch_conv_decode<IO, 3>(a, cols, st);
    return varlen ? launch_conv_varlen<IO, 4>(a, cols, st) : launch_conv_decode<IO, 4>(a, cols, st);
}

int check_conv(const kda_conv_params* p)
{
    if (!p) return KDA_ERR_INVALID_ARGUMENT;
    if (p->conv_kernel < 2 || p->conv_kernel > 4) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (p->channels <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (p->channels % 8 != 0 || p->channels > (1 << 20)) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if (!known_dtype(p->io_dtype) || p->num_slots <= 0) return KDA_ERR_INVALID_ARGUMENT;
    return check_ptrs({p->conv_weight});
}

int conv_call(const kda_conv_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const void* x,
              const int32_t* slots, void* conv_state, void* y, int32_t* dev_status, bool varlen, cudaStream_t stream)
{
    int rc;
    if ((rc = check_ptrs({x, conv_state, y})) != KDA_OK || (rc = check_opt(slots)) != KDA_OK) return rc;
    const size_t row = (size_t)p->channels * io_size(p->io_dtype);
    const size_t state = (size_t)p->num_slots * (p->conv_kernel - 1) * row;
    if (overlap(x, T * row, y, T * row) || overlap(conv_state, state, y, T * row) || overlap(conv_state, state, x, T * row))
        return KDA_ERR_INVALID_ARGUMENT;
    const void* lists[3] = {p->conv_weight, cu_seqlens, slots};
    const size_t size[3] = {row / io_size(p->io_dtype) * p->conv_kernel * sizeof(float), ((size_t)N + 1) * sizeof(int32_t),
                            (size_t)N * sizeof(int32_t)};
    for (int i = 0; i < 3; ++i)
        if (overlap(y, T * row, lists[i], size[i]) || overlap(conv_state, state, lists[i], size[i]))
            return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    ConvArgs a;
    a.C = p->channels;
    a.N = N;
    a.T = T;
    a.num_slots = p->num_slots;
    a.cu_seqlens = cu_seqlens;
    a.x = x;
    a.w = p->conv_weight;
    a.slots = slots;
    a.state = conv_state;
    a.y = y;
    a.dev_status = dev_status;
    const cudaError_t e = p->io_dtype == KDA_DTYPE_BF16 ? launch_conv<__nv_bfloat16>(a, p->conv_kernel, varlen, stream)
                                                        : launch_conv<float>(a, p->conv_kernel, varlen, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

// ------------------------------------------------------------ block norms

struct NormArgs {
    int D, post, act;
    long long rows;
    float scale, eps, inv_d;
    const void* y;
    const void* gate;
    const void* res;
    const float* post_w;
    const float* pre_w;
    void* h;
    void* x;
};

// The row's values in fp32 across a group of threads, VPT vectors of eight
// each; sum() adds over the group.  One pass: every value is read once, kept in registers
// through both norms and written once.  Bound: HBM.  16384 rows of 4096 values
// (bf16, fp32 residual stream, both outputs) take 135 us, 6960 GB/s; the post norm and
// gate of 2048 heads' rows of 128 3.2 us, the launch's time.
template <typename IO, typename RES, int VPT, class Sum>
__device__ __forceinline__ void norm_row(const NormArgs& a, long long row, int first, int step, bool live, Sum&& sum)
{
    const int nv = a.D / 8;
    const size_t base = (size_t)row * a.D;
    const IO* y = static_cast<const IO*>(a.y) + base;
    const IO* g = static_cast<const IO*>(a.gate) + base;
    const RES* res = static_cast<const RES*>(a.res) + base;
    Vec8<IO> yv[VPT], gv[VPT];
    Vec8<RES> rv[VPT];
    // every load of the row first
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        const bool in = live && v < nv;
        if (in) yv[j].load(y + v * 8);
        else yv[j].zero();
        if (a.act != KDA_NORM_GATE_NONE && in) gv[j].load(g + v * 8);
        else gv[j].zero();
        if (a.res && in) rv[j].load(res + v * 8);
        else rv[j].zero();
    }
    float t[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        yv[j].get(t[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(t[j][i], t[j][i], ss);
    }
    const float post = a.post ? rsqrtf(sum(ss) * a.inv_d + a.eps) : 1.f;
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        const bool in = live && v < nv;
        float w[8], gx[8], rx[8];
        if (a.post && a.post_w && in) {
            Vec8<float> wv;
            wv.load(a.post_w + v * 8);
            wv.get(w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
        gv[j].get(gx);
        rv[j].get(rx);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float z = t[j][i] * post * w[i];
            if (a.act == KDA_NORM_GATE_SIGMOID) z *= sigmoidf_(gx[i]);
            else if (a.act == KDA_NORM_GATE_SILU) z *= siluf_(gx[i]);
            z *= a.scale;
            if (a.res) z += rx[i];
            t[j][i] = in ? z : 0.f;
            ss = fmaf(t[j][i], t[j][i], ss);
        }
        if (a.h && in) {
            Vec8<RES> o;
            o.set(t[j]);
            o.store(static_cast<RES*>(a.h) + base + v * 8);
        }
    }
    if (!a.x) return;
    const float pre = rsqrtf(sum(ss) * a.inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if (!(live && v < nv)) continue;
        float w[8];
        if (a.pre_w) {
            Vec8<float> wv;
            wv.load(a.pre_w + v * 8);
            wv.get(w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = t[j][i] * pre * w[i];
        Vec8<IO> ov;
        ov.set(o);
        ov.store(static_cast<IO*>(a.x) + base + v * 8);
    }
}

// Rows of up to 512 values: a power of two of lanes for each (a CTA for a row of 1024
// values does as well as a warp, 134 and 136 us for 65536 of them).
template <typename IO, typename RES, int VPT>
__global__ void __launch_bounds__(128) norm_warp_kernel(const NormArgs a, int lanes)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, per_warp = 32 / lanes;
    const long long row = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * per_warp + lane / lanes;
    norm_row<IO, RES, VPT>(a, row < a.rows ? row : 0, lane % lanes, lanes, row < a.rows, [&](float s) {
        for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    });
}

// Longer rows: a CTA for each, two vectors a thread (four at rows of 4096 values: 141 us
// against 135; at 16384 values 174 against 168).
template <typename IO, typename RES>
__global__ void __launch_bounds__(1024) norm_block_kernel(const NormArgs a)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ float part[2][32];
    int turn = 0;
    norm_row<IO, RES, 2>(a, blockIdx.x, threadIdx.x, blockDim.x, true, [&](float s) {
        s = warp_sum(s);
        float* p = part[turn++];
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = s;
        __syncthreads();
        s = 0.f;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += p[w];
        return s;
    });
}

template <typename IO, typename RES> cudaError_t launch_norm(const NormArgs& a, cudaStream_t st)
{
    const int nv = a.D / 8;
    if (nv <= 64) {
        int lanes = 1;
        while (lanes < nv && lanes < 32) lanes <<= 1;
        const long long per_cta = 4 * (32 / lanes);
        const unsigned g = (unsigned)((a.rows + per_cta - 1) / per_cta);
        if (nv <= 32) return launch_dependent(norm_warp_kernel<IO, RES, 1>, g, 128, 0, st, a, lanes);
        return launch_dependent(norm_warp_kernel<IO, RES, 2>, g, 128, 0, st, a, lanes);
    }
    return launch_dependent(norm_block_kernel<IO, RES>, (unsigned)a.rows, ((nv + 1) / 2 + 31) / 32 * 32, 0, st, a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

KDA_API int kda_conv_varlen(const kda_conv_params* p, const int32_t* cu_seqlens, int32_t N, int32_t T, const void* x,
                            const int32_t* slots, void* conv_state, void* y, int32_t* dev_status,
                            cudaStream_t stream)
{
    int rc = check_conv(p);
    if (rc != KDA_OK) return rc;
    // tiles are counted by index, and the search for one looks up to 31 sequences past the last
    if (N < 0 || T < 0 || T > KDA_MAX_ROWS || (int64_t)N + T / 16 > KDA_MAX_ROWS) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0 || T == 0) return KDA_OK;
    if ((rc = check_ptrs({cu_seqlens})) != KDA_OK) return rc;
    return conv_call(p, cu_seqlens, N, T, x, slots, conv_state, y, dev_status, true, stream);
}

KDA_API int kda_conv_decode(const kda_conv_params* p, int32_t B, const void* x, const int32_t* slots,
                            void* conv_state, void* y, int32_t* dev_status, cudaStream_t stream)
{
    int rc = check_conv(p);
    if (rc != KDA_OK) return rc;
    if (B < 0 || B > KDA_MAX_ROWS) return KDA_ERR_INVALID_ARGUMENT;
    if (B == 0) return KDA_OK;
    return conv_call(p, nullptr, B, B, x, slots, conv_state, y, dev_status, false, stream);
}

KDA_API int kda_block_norm(const kda_norm_params* p, int64_t rows, const void* y, const void* gate,
                           const void* residual, void* h_out, void* x_out, cudaStream_t stream)
{
    if (!p || rows < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (p->dim <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (p->dim % 8 != 0 || p->dim > 16384) return KDA_ERR_UNSUPPORTED_GEOMETRY;
    if ((p->post_norm != 0 && p->post_norm != 1) || p->gate_act < KDA_NORM_GATE_NONE || p->gate_act > KDA_NORM_GATE_SILU)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(p->residual_scale) || !(std::isfinite(p->norm_eps) && p->norm_eps >= 0.0f))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!known_dtype(p->io_dtype) || !known_dtype(p->res_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    int rc;
    if ((rc = check_opt(p->post_weight)) != KDA_OK || (rc = check_opt(p->pre_weight)) != KDA_OK) return rc;
    if (rows == 0) return KDA_OK;
    if (rows > INT32_MAX) return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_ptrs({y})) != KDA_OK) return rc;
    if (p->gate_act != KDA_NORM_GATE_NONE && (rc = check_ptrs({gate})) != KDA_OK) return rc;
    if ((rc = check_opt(residual)) != KDA_OK || (rc = check_opt(h_out)) != KDA_OK || (rc = check_opt(x_out)) != KDA_OK)
        return rc;
    if (!h_out && !x_out) return KDA_ERR_INVALID_ARGUMENT;
    if (p->gate_act == KDA_NORM_GATE_NONE) gate = nullptr;
    const size_t io = (size_t)rows * p->dim * io_size(p->io_dtype), rs = (size_t)rows * p->dim * io_size(p->res_dtype);
    // in place is the very buffer, of one type; anything else that overlaps is refused
    auto clash = [](const void* out, size_t no, const void* in, size_t ni) {
        return overlap(out, no, in, ni) && !(out == in && no == ni);
    };
    if (clash(h_out, rs, y, io) || clash(h_out, rs, gate, io) || clash(h_out, rs, residual, rs) ||
        clash(x_out, io, y, io) || clash(x_out, io, gate, io) || clash(x_out, io, residual, rs) ||
        overlap(h_out, rs, x_out, io))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const float* w : {p->post_weight, p->pre_weight})
        if (overlap(h_out, rs, w, p->dim * sizeof(float)) || overlap(x_out, io, w, p->dim * sizeof(float)))
            return KDA_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != KDA_OK) return rc;
    NormArgs a;
    a.D = p->dim;
    a.post = p->post_norm;
    a.act = p->gate_act;
    a.rows = rows;
    a.scale = p->residual_scale;
    a.eps = p->norm_eps;
    a.inv_d = 1.0f / (float)p->dim;
    a.y = y;
    a.gate = gate;
    a.res = residual;
    a.post_w = p->post_weight;
    a.pre_w = p->pre_weight;
    a.h = h_out;
    a.x = x_out;
    const bool iob = p->io_dtype == KDA_DTYPE_BF16, rsb = p->res_dtype == KDA_DTYPE_BF16;
    const cudaError_t e = iob && rsb ? launch_norm<__nv_bfloat16, __nv_bfloat16>(a, stream)
                        : iob        ? launch_norm<__nv_bfloat16, float>(a, stream)
                        : rsb        ? launch_norm<float, __nv_bfloat16>(a, stream)
                                     : launch_norm<float, float>(a, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // extern "C"
