// What the attention kernels over a paged cache share: types of the matrix products, the list of units of
// work and its runs, the workspace of their pieces, and the launch that joins them.
#pragma once

#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256, kWaves = 4, kTile = 32, kUnit = kWaves * kTile;
constexpr int kMaxWorkers = 512;   // work-groups of a launch; each leaves at most two pieces
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(Bf16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(Fp16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(Bf16, float a, float b)
{
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t pack2(Fp16, float a, float b)
{
    const f16x2 r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// Two e4m3 codes (the low or the high half of a word) as 16-bit values, exactly.
template <bool HI>
__device__ __forceinline__ uint32_t from_e4m3(Bf16, uint32_t w)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}
template <bool HI>
__device__ __forceinline__ uint32_t from_e4m3(Fp16, uint32_t w)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// Largest value, and sum, over the four lanes that share lane % 16.
__device__ __forceinline__ float max4(float x)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    u = __builtin_bit_cast(uint32_t, x);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)s[0]), __builtin_bit_cast(float, (uint32_t)s[1]));
}
__device__ __forceinline__ float sum4(float x)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    u = __builtin_bit_cast(uint32_t, x);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}

__device__ __forceinline__ int64_t read64(int64_t v, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane((int)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// ---- the list of units ---------------------------------------------------------------------------

struct Span {
    int32_t n, lo, base;   // positions lo <= j < n; the first unit starts at base
    uint32_t units;
};

__device__ __forceinline__ Span span_of(const AttentionArgs &a, int b)
{
    const int32_t len = max(a.lens[b], 0);
    Span s;
    s.n = min(len, a.max_pages * a.page_size);
    s.lo = a.window ? max(len - a.window, 0) : 0;
    s.base = s.lo & ~(kUnit - 1);
    s.units = s.n > s.lo ? ((uint32_t)(s.n - s.base) + kUnit - 1) / kUnit : 1;
    return s;
}

// Where a run of units starts, and how long the runs are. The host has made sure that there are fewer
// than 2^31 units.
struct Place {
    uint32_t per, u0, u1;   // units per work-group, this work-group's run
    uint32_t first;         // units of a request before request b, for one of its heads
    int b;
};

// Finds the request that holds this work-group's first unit. Up to 64 requests: a running sum in every
// wave (no barrier; one request of 1100 tokens 6.8 -> 5.6 us). More: every thread sums a run of
// requests, those sums are scanned through LDS, and the request is looked for in its run. `groups`:
// (KV head, 16 query heads) pairs per request.
__device__ __forceinline__ Place find_run(const AttentionArgs &a, uint32_t groups, uint32_t *before)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Place p;
    if (a.B <= 64) {
        const uint32_t units = lane < a.B ? span_of(a, lane).units : 0;
        uint32_t s = units;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t t = __shfl_up(s, d);
            if (lane >= d)
                s += t;
        }
        const uint32_t total = __builtin_amdgcn_readlane(s, 63) * groups;
        p.per = (total + gridDim.x - 1) / gridDim.x;
        p.u0 = min(blockIdx.x * p.per, total);
        p.u1 = min(p.u0 + p.per, total);
        p.b = 63 - __builtin_clzll(__ballot(lane < a.B && (s - units) * groups <= p.u0) | 1);
        p.first = __builtin_amdgcn_readlane(s - units, p.b);
        return p;
    }
    __shared__ uint32_t wave_sum[kWaves];
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b)
        sum += span_of(a, b).units;
    uint32_t s = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t t = __shfl_up(s, d);
        if (lane >= d)
            s += t;
    }
    if (lane == 63)
        wave_sum[wave] = s;
    __syncthreads();
    uint32_t total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave)
            s += wave_sum[w];
        total += wave_sum[w];
    }
    before[tid] = s - sum;
    __syncthreads();
    total *= groups;
    p.per = (total + gridDim.x - 1) / gridDim.x;
    p.u0 = min(blockIdx.x * p.per, total);
    p.u1 = min(p.u0 + p.per, total);
    int r = 0;
    for (int step = kThreads / 2; step; step >>= 1)
        if ((r + step) * per < a.B && before[r + step] * groups <= p.u0)
            r += step;
    p.b = r * per;
    p.first = before[r];
    while (p.b + 1 < a.B) {
        const uint32_t next = p.first + span_of(a, p.b).units;
        if (next * groups > p.u0)
            break;
        p.first = next;
        ++p.b;
    }
    return p;
}

// One (request, KV head, 16 query heads).
struct Head {
    int b, kv, h0, heads;   // first query head, and how many
};

__device__ __forceinline__ Head head_of(const AttentionArgs &a, int b, int group)
{
    const int share = a.Hq / a.Hkv, parts = (share + 15) / 16;
    Head h;
    h.b = b;
    h.kv = group / parts;
    const int part = group - h.kv * parts;
    h.h0 = h.kv * share + part * 16;
    h.heads = min(16, share - part * 16);
    return h;
}

// The workspace: sums [16][D] of every piece, then their maxima and sums of weights [16][2], then for
// each work-group what it holds the end of and does not hold the start of.
struct Ending {
    int32_t b, group, from;   // request (or -1), head, and the work-group that holds the start
};
__device__ __forceinline__ float *piece_sums(const AttentionArgs &a, int i) { return a.work + (int64_t)i * 16 * a.dim; }
__device__ __forceinline__ float *piece_stats(const AttentionArgs &a, int i)
{
    return a.work + (int64_t)2 * kMaxWorkers * 16 * a.dim + i * 32;
}
__device__ __forceinline__ Ending *endings(const AttentionArgs &a)
{
    return (Ending *)(a.work + (int64_t)2 * kMaxWorkers * 16 * (a.dim + 2));
}

template <class Type>
__device__ __forceinline__ void store_out(const AttentionArgs &a, int64_t b, int h, int d, f32x4 o)
{
    u32x2 r;
    r[0] = pack2(Type(), o[0], o[1]);
    r[1] = pack2(Type(), o[2], o[3]);
    *(u32x2 *)((uint16_t *)a.out + b * a.ldo + h * a.hso + d) = r;
}

// ---- one tile's operands -------------------------------------------------------------------------

// Words of 16-bit values per lane and V row; a row is loaded in parts of 16 lanes each:
// 64 dims (4 per lane), 96 (4 and 2), 128 (8), 192 (8 and 4), 256 (8 and 8).
template <int D>
struct Parts {
    static constexpr int words = D / 32;
    static constexpr int first = D >= 128 ? 8 : 4;            // dims per lane of the first part
    static constexpr int second = D / 16 - first;             // and of the second, or 0
    // dim of local value j of lane i
    static __device__ __forceinline__ int dim(int i, int j)
    {
        return j < first ? first * i + j : 16 * first + second * i + (j - first);
    }
};

// N 16-bit values (N / 2 words) from memory, or N e4m3 codes (N / 4 words, at least one).
template <int N, bool E4M3>
__device__ __forceinline__ void load_part(const uint8_t *p, uint32_t *r)
{
    constexpr int bytes = E4M3 ? N : 2 * N;
    if constexpr (bytes == 16) {
        const u32x4 x = __builtin_nontemporal_load((const u32x4 *)p);
        r[0] = x[0]; r[1] = x[1]; r[2] = x[2]; r[3] = x[3];
    } else if constexpr (bytes == 8) {
        const u32x2 x = __builtin_nontemporal_load((const u32x2 *)p);
        r[0] = x[0]; r[1] = x[1];
    } else if constexpr (bytes == 4) {
        r[0] = *(const uint32_t *)p;
    } else {
        static_assert(bytes == 2, "parts are 2 to 16 bytes");
        r[0] = *(const uint16_t *)p;
    }
}

// K rows as the first operand of S^T = K Q^T: lane % 16 is the position, and a contraction of 32 dims
// takes 8 from each of the four lanes of a position. bfloat16 / float16: dims 32c + 8g. e4m3: one
// 16-byte load serves two contractions (dims 64 (c / 2) + 16 g + 8 (c % 2)), the last 32 of 96
// dims come in 8-byte loads.
template <int D, bool E4M3>
struct KeyDims {
    static constexpr int chunks = D / 32, paired = E4M3 ? D / 64 * 2 : 0;
    static __device__ __forceinline__ int dim(int c, int g)
    {
        return c < paired ? 64 * (c / 2) + 16 * g + 8 * (c % 2) : 32 * c + 8 * g;
    }
};

// ---- the second launch ---------------------------------------------------------------------------

// Joins the pieces of a (request, head) that several work-groups share; the one that holds its end
// has left a note. A thread sums four dims of one head over every `parts`-th piece, with the maximum
// running along; the parts are then joined in order. (With the notes instead of another search for
// the run, and the pieces spread over threads, one request of 131000 tokens went from 149 to 115 us.)
constexpr int kJoinThreads = 512;

struct Sum {
    float m, l;
    f32x4 o;
    __device__ __forceinline__ void add(float m2, float l2, f32x4 o2)
    {
        const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
        const float f = __builtin_amdgcn_exp2f(m - ref), f2 = __builtin_amdgcn_exp2f(m2 - ref);
        m = top;
        l = l * f + l2 * f2;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = o[e] * f + o2[e] * f2;
    }
};

template <class Type>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttentionArgs a)
{
    __shared__ __align__(16) f32x4 part_o[kJoinThreads];
    __shared__ f32x2 part_ml[kJoinThreads];
    const Ending end = endings(a)[blockIdx.x];
    if (end.b < 0)
        return;
    const int tid = threadIdx.x, to = (int)blockIdx.x;
    const Head head = head_of(a, end.b, end.group);
    const float v_scale = a.e4m3 && a.v_scale ? a.v_scale[head.kv] : 1.0f;
    const int quads = a.dim / 4, items = head.heads * quads;
    const int parts = min(max(kJoinThreads / items, 1), to - end.from + 1);
    for (int i0 = 0; i0 < items; i0 += kJoinThreads) {   // more than once for 16 heads of 192 and 256 dims
        const int part = i0 ? 0 : tid / items, x = i0 + tid - part * items;
        const bool mine = x < items && part < parts;
        const int h = x / quads, d = (x - h * quads) * 4;
        Sum sum{-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
        if (mine) {
#pragma unroll 4
            for (int w = end.from + part; w <= to; w += parts) {
                const int piece = 2 * w + (w == end.from);
                const f32x2 ml = *(const f32x2 *)(piece_stats(a, piece) + 2 * h);
                sum.add(ml[0], ml[1], *(const f32x4 *)(piece_sums(a, piece) + h * a.dim + d));
            }
            if (part > 0) {
                part_ml[tid] = f32x2{sum.m, sum.l};
                part_o[tid] = sum.o;
            }
        }
        __syncthreads();
        if (mine && part == 0) {
            for (int p = 1; p < parts; ++p)
                sum.add(part_ml[tid + p * items][0], part_ml[tid + p * items][1], part_o[tid + p * items]);
            const float f = sum.l == 0.0f ? 0.0f : v_scale / sum.l;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum.o[e] = sum.l == 0.0f ? 0.0f : sum.o[e] * f;
            store_out<Type>(a, end.b, head.h0 + h, d, sum.o);
            if (d == 0 && a.lse)
                a.lse[(int64_t)end.b * a.Hq + head.h0 + h] =
                    sum.l == 0.0f ? -INFINITY : (sum.m + __builtin_amdgcn_logf(sum.l)) * kLn2;
        }
        __syncthreads();
    }
}

}  // namespace

}  // namespace w4a16
