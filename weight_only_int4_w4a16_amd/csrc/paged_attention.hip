// Attention of one new token per request over a paged key-value cache, for gfx950:
//   s_j = scale * q . k_j,   out = sum_j e^{s_j} v_j / sum_j e^{s_j}   over the cached positions j.
//
// Every cached row is read once and used for the query heads that share its KV head (up to 16 at a
// time), so the cache's bytes bound the kernel: 4 flops per value, head and byte pair are far from
// what the matrix units can do, and they are used only because 16 heads at a time cost nothing there.
//
// Split. The work is the list of all units, a unit being 128 positions of one request and KV head (a
// request without positions has one empty unit). The list is cut into equal runs, one per
// work-group: lengths live on the device, so every work-group makes the running sum of the units
// itself and finds its run in it. Ragged batches, one long request and many short ones are then the
// same case. A run crosses from one (request, head) to the next; a piece that is not the whole of its
// (request, head) leaves its sums in the workspace, and a second launch joins them in a fixed order.
//
// A wave takes every fourth tile of 32 positions. With MFMA 16x16x32 the scores are computed
// transposed, S^T = K Q^T: a lane then holds one head (lane % 16) and the positions 4g..4g+3 and
// 16 + 4g..16 + 4g + 3 (g = lane / 16) of the tile. O^T = V^T P^T contracts over positions, whose
// order inside a contraction is free, so those eight probabilities are the second operand as they are,
// and V rows of the same eight positions are the first: each lane loads the same dims of eight rows
// (whole rows per 16 lanes) and pairs rows up with byte permutes. No value crosses lanes but the maximum
// of a tile.
//
// The loads of a tile's V and of the next tile's K are in flight during the arithmetic: 8 to 16 KB
// for each of 8 waves per CU (bfloat16, dim 128). More work-groups per CU (3 or 4, with fewer registers
// each) are slower (64 ragged requests of up to 8192 positions 152 -> 175 and 269 us).
// They are streaming loads: nothing is read twice, and kept lines only push others out (the same requests
// 171 -> 152 us before the last steps).
//
// Measured, 8 KV heads of 128: those 64 requests, 8 query heads to a KV head, 144 us in all, 140 of them
// here (6.15 TB/s, where a plain streaming read of 4 GiB reaches 6.3); 48 requests of 5000 positions as e4m3 27 us
// here and 5 us joining; one request of 131000 positions 96 and 8 us (5.6 TB/s); one of 1100
// positions 5.8 and 4.4 us, which is latency: lengths, page table, rows, the join of four waves, and all
// that once more for the second launch.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256, kWaves = 4, kTile = 32, kUnit = kWaves * kTile;
constexpr int kMaxWorkers = 512;   // work-groups of a launch; each leaves at most two pieces
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// Weights are 2^(score - reference), scores in powers of two, and the reference is this much below the largest
// score so far: float16 weights then keep their 11 bits down to 2^-29 of the largest one. (With 0 they lost them
// from 2^-14 on, and 18 nats behind a position of little value all others were gone from the sum.)
template <class Type>
constexpr float kHeadroom = __is_same(Type, Fp16) ? 15.0f : 0.0f;

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

// The words of one V row as they come from memory, and as 16-bit values.
template <class Type, int D, bool E4M3>
struct Row {
    static constexpr int first = Parts<D>::first, second = Parts<D>::second;
    static constexpr int head = E4M3 ? first / 4 : first / 2;
    static constexpr int raw = head + (second ? (E4M3 ? (second + 3) / 4 : second / 2) : 0);
    uint32_t w[raw];
    // p: the row's lane address of the first part (first * i dims in); q: of the second
    __device__ __forceinline__ void load(const uint8_t *p, const uint8_t *q)
    {
        load_part<first, E4M3>(p, w);
        if constexpr (second > 0)
            load_part<second, E4M3>(q, w + head);
    }
    __device__ __forceinline__ uint32_t word(int x) const   // values 2x and 2x + 1
    {
        if constexpr (!E4M3)
            return w[x];
        else
            return x % 2 ? from_e4m3<true>(Type(), w[x / 2]) : from_e4m3<false>(Type(), w[x / 2]);
    }
};

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

template <class Type, int D, bool E4M3>
struct Keys {   // one half tile: 16 positions
    static constexpr int chunks = D / 32, words = E4M3 ? 2 : 4;
    uint32_t w[chunks][words];
    __device__ __forceinline__ void load(const uint8_t *p, int g)
    {
        typedef KeyDims<D, E4M3> KD;
#pragma unroll
        for (int c = 0; c < chunks; ++c) {
            if constexpr (!E4M3) {
                const u32x4 x = __builtin_nontemporal_load((const u32x4 *)(p + 2 * KD::dim(c, g)));
                w[c][0] = x[0]; w[c][1] = x[1]; w[c][2] = x[2]; w[c][3] = x[3];
            } else if (c < KD::paired) {
                if (c % 2 == 0) {
                    const u32x4 x = __builtin_nontemporal_load((const u32x4 *)(p + KD::dim(c, g)));
                    w[c][0] = x[0]; w[c][1] = x[1]; w[c + 1][0] = x[2]; w[c + 1][1] = x[3];
                }
            } else {
                const u32x2 x = *(const u32x2 *)(p + KD::dim(c, g));
                w[c][0] = x[0]; w[c][1] = x[1];
            }
        }
    }
    __device__ __forceinline__ u32x4 operand(int c) const
    {
        u32x4 r;
        if constexpr (!E4M3) {
            r[0] = w[c][0]; r[1] = w[c][1]; r[2] = w[c][2]; r[3] = w[c][3];
        } else {
            r[0] = from_e4m3<false>(Type(), w[c][0]);
            r[1] = from_e4m3<true>(Type(), w[c][0]);
            r[2] = from_e4m3<false>(Type(), w[c][1]);
            r[3] = from_e4m3<true>(Type(), w[c][1]);
        }
        return r;
    }
};

// Addresses of a tile's rows. WHOLE: the page size is a multiple of 16, so each half tile lies in one
// page and its address is uniform; a lane holds the offsets of one half tile, for 32 tiles of the
// wave at a time. Otherwise a lane looks up one position of the tile, and rows are found by shuffles.
// Positions that are not read (outside lo..n-1, or on a page that is none) have offset 0, which is in
// the cache, and their bit of `live` is 0.
template <bool E4M3, bool WHOLE>
struct Rows {
    int64_t k, v;        // byte offsets: this lane's half tile (WHOLE), or this lane's position
    uint64_t fine;       // lanes whose page is one of the cache
    uint32_t live;       // bit i: position i of the tile is read
    int64_t k0, k1, v0, v1;   // WHOLE: offsets of the two half tiles

    __device__ __forceinline__ void lookup(const AttentionArgs &a, const Head &h, int64_t j, bool inside)
    {
        constexpr int size = E4M3 ? 1 : 2;
        const uint32_t at = (uint32_t)j / (uint32_t)a.page_size, slot = (uint32_t)j - at * (uint32_t)a.page_size;
        int32_t page = -1;
        if (inside)
            page = a.table[h.b * a.row_stride + at];
        const bool ok = page >= 0 && page < a.num_pages;
        k = ok ? (page * a.k_page + slot * a.k_slot) * size : 0;
        v = ok ? (page * a.v_page + slot * a.v_slot) * size : 0;
        fine = __ballot(ok);
    }
    // Tile number `i` of the wave, at position j0 = start + i * kUnit.
    __device__ __forceinline__ void go(const AttentionArgs &a, const Head &h, const Span &s, int start, int i)
    {
        const int lane = threadIdx.x & 63;
        const int64_t j0 = (int64_t)start + (int64_t)i * kUnit;
        const int64_t below = s.lo - j0, above = s.n - j0;   // positions of the tile: below <= . < above
        uint32_t in = above >= 32 ? ~0u : above <= 0 ? 0u : (1u << above) - 1;
        in &= below <= 0 ? ~0u : below >= 32 ? 0u : ~0u << below;
        if constexpr (WHOLE) {
            if ((i & 31) == 0) {
                const int64_t j = j0 + (int64_t)(lane >> 1) * kUnit + (lane & 1) * 16;
                lookup(a, h, j, j < s.n && j + 16 > s.lo);
            }
            const int at = 2 * (i & 31);
            k0 = read64(k, at);
            k1 = read64(k, at + 1);
            v0 = read64(v, at);
            v1 = read64(v, at + 1);
            const uint32_t two = (uint32_t)(fine >> at);
            live = in & ((two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u));
        } else {
            const int64_t j = j0 + (lane & 31);
            lookup(a, h, j, (in >> (lane & 31)) & 1);
            live = (uint32_t)fine;
        }
    }
};

__device__ __forceinline__ int64_t shuffle64(int64_t v, int lane)
{
    const uint32_t lo = __shfl((int)v, lane), hi = __shfl((int)(v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

template <class Type, bool E4M3, int D, bool WHOLE>
__global__ __launch_bounds__(kThreads, E4M3 || D <= 128 ? 2 : 1) void attention_kernel(AttentionArgs a)
{
    constexpr int size = E4M3 ? 1 : 2;
    typedef Parts<D> P;
    constexpr int pad = D + 4;
    __shared__ __align__(16) float sums[kWaves][16][pad];   // the scan's sums before that
    __shared__ float tops[kWaves][16], totals[kWaves][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int share = a.Hq / a.Hkv, groups = a.Hkv * ((share + 15) / 16);
    const Place place = find_run(a, groups, (uint32_t *)sums);
    uint32_t u = place.u0;
    if (u >= place.u1) {
        if (tid == 0)
            endings(a)[blockIdx.x].b = -1;
        return;
    }
    int b = place.b;
    Span span = span_of(a, b);
    const uint32_t inside = u - place.first * groups;
    int group = (int)(inside / span.units);
    uint32_t t0 = inside - group * span.units;
    if (tid == 0) {
        const uint32_t begin = u - t0;
        const bool ends = t0 > 0 && begin + span.units <= place.u1;
        endings(a)[blockIdx.x] = Ending{ends ? b : -1, group, (int)(begin / place.per)};
    }

    // This lane's share of a row, in bytes.
    const uint32_t k_lane = (uint32_t)(col * a.k_slot * size), v_lane = (uint32_t)(4 * g * a.v_slot * size);
    const uint32_t first = P::first * col * size, second = (16 * P::first + P::second * col) * size;

    while (u < place.u1) {
        const uint32_t count = min(place.u1 - u, span.units - t0);
        const Head head = head_of(a, b, group);
        const uint8_t *kb = (const uint8_t *)a.k + head.kv * a.k_head * size;
        const uint8_t *vb = (const uint8_t *)a.v + head.kv * a.v_head * size;
        const int start = span.base + (int)(t0 * kUnit) + wave * kTile;
        // tiles of this wave: the last unit may end before this wave's tile of it
        int tiles = (int)count;
        if (tiles && (int64_t)start + (int64_t)(tiles - 1) * kUnit >= span.n)
            --tiles;

        u32x4 q[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            q[c] = u32x4{0, 0, 0, 0};
            if (col < head.heads)
                q[c] = *(const u32x4 *)((const uint16_t *)a.q + b * a.ldq + (head.h0 + col) * a.hsq +
                                        KeyDims<D, E4M3>::dim(c, g));
        }
        const float to_log2 = a.scale * kLog2e * (E4M3 && a.k_scale ? a.k_scale[head.kv] : 1.0f);

        Keys<Type, D, E4M3> keys[2];
        Row<Type, D, E4M3> rows[8];
        Rows<E4M3, WHOLE> r;
        auto load_keys = [&]() {
            if constexpr (WHOLE) {
                keys[0].load(kb + r.k0 + k_lane, g);
                keys[1].load(kb + r.k1 + k_lane, g);
            } else {
                keys[0].load(kb + shuffle64(r.k, col), g);
                keys[1].load(kb + shuffle64(r.k, 16 + col), g);
            }
        };
        auto load_rows = [&]() {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint8_t *p;
                if constexpr (WHOLE)
                    p = vb + (e < 4 ? r.v0 : r.v1) + (e & 3) * a.v_slot * size + v_lane;
                else
                    p = vb + shuffle64(r.v, (e < 4 ? 0 : 12) + 4 * g + e);
                rows[e].load(p + first, p + second);
            }
        };

        f32x4 o[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float top = -INFINITY, total = 0.0f;   // total: this lane's positions only, until the end
        if (tiles) {
            r.go(a, head, span, start, 0);
            load_keys();
        }
        for (int i = 0; i < tiles; ++i) {
            load_rows();
            const uint32_t live = r.live;
            __builtin_amdgcn_sched_barrier(0);
            f32x4 s[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                s[half] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    s[half] = mfma(Type(), keys[half].operand(c), q[c], s[half]);
            }
            if (i + 1 < tiles) {
                r.go(a, head, span, start, i + 1);
                load_keys();
            }
            __builtin_amdgcn_sched_barrier(0);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = s[e >> 2][e & 3] * to_log2;
            if (live != ~0u) {   // positions that are not read: no weight, and no value either
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!((live >> ((e < 4 ? 0 : 12) + 4 * g + e)) & 1)) {
                        x[e] = -INFINITY;
#pragma unroll
                        for (int w = 0; w < Row<Type, D, E4M3>::raw; ++w)
                            rows[e].w[w] = 0;
                    }
            }
            float m = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e)
                m = fmaxf(m, x[e]);
            m = fmaxf(max4(m) - kHeadroom<Type>, top);
            const float ref = m == -INFINITY ? 0.0f : m;   // nothing seen yet: every weight is 0
            const float fade = __builtin_amdgcn_exp2f(top - ref);
            top = m;
            total *= fade;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __builtin_amdgcn_exp2f(x[e] - ref);
                total += x[e];
            }
            // The weights, at most 2^kHeadroom, are rounded to the activations' type for the matrix
            // product (their sum is not): what a float32 product would cost is 8 times the MFMA time.
            u32x4 p;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = pack2(Type(), x[2 * e], x[2 * e + 1]);
#pragma unroll
            for (int w = 0; w < P::words; ++w) {
                u32x4 lo, hi;   // values 2w and 2w + 1 of the eight rows
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x0 = rows[2 * e].word(w), x1 = rows[2 * e + 1].word(w);
                    lo[e] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                    hi[e] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[2 * w][k] *= fade;
                    o[2 * w + 1][k] *= fade;
                }
                o[2 * w] = mfma(Type(), lo, p, o[2 * w]);
                o[2 * w + 1] = mfma(Type(), hi, p, o[2 * w + 1]);
            }
        }

        // Join the four waves in LDS. A lane holds, of head col, dims of V lane 4g + k (k < 4).
        total = sum4(total);
        __syncthreads();   // the scan's sums, or the previous piece's, have been read
        if (g == 0) {
            tops[wave][col] = top;
            totals[wave][col] = total;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < D / 16; j += 2)
                *(f32x2 *)&sums[wave][col][P::dim(4 * g + k, j)] = f32x2{o[j][k], o[j + 1][k]};
        __syncthreads();
        const bool whole = t0 == 0 && count == span.units;
        const int piece = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
        const float v_scale = E4M3 && a.v_scale ? a.v_scale[head.kv] : 1.0f;
        for (int x = tid; x < head.heads * (D / 4); x += kThreads) {
            const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
            float m = tops[0][h];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                m = fmaxf(m, tops[w][h]);
            const float ref = m == -INFINITY ? 0.0f : m;
            float l = 0.0f;
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(tops[w][h] - ref);
                l = fmaf(totals[w][h], f, l);
                const f32x4 y = *(const f32x4 *)&sums[w][h][d];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = fmaf(y[e], f, sum[e]);
            }
            if (whole) {
                const float f = l == 0.0f ? 0.0f : v_scale / l;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = l == 0.0f ? 0.0f : sum[e] * f;
                store_out<Type>(a, b, head.h0 + h, d, sum);
                if (d == 0 && a.lse)
                    a.lse[(int64_t)b * a.Hq + head.h0 + h] =
                        l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
            } else {
                *(f32x4 *)(piece_sums(a, piece) + h * D + d) = sum;
                if (d == 0)
                    *(f32x2 *)(piece_stats(a, piece) + 2 * h) = f32x2{m, l};
            }
        }

        u += count;
        t0 = 0;
        if (++group == groups) {
            group = 0;
            if (++b < a.B)
                span = span_of(a, b);
        }
    }
}

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

template <class Type, bool E4M3, int D>
void attention_of(const AttentionArgs &a, bool whole, int workers, hipStream_t stream)
{
    whole ? attention_kernel<Type, E4M3, D, true><<<dim3(workers), dim3(kThreads), 0, stream>>>(a)
          : attention_kernel<Type, E4M3, D, false><<<dim3(workers), dim3(kThreads), 0, stream>>>(a);
}

template <class Type, bool E4M3>
void attention_dim(const AttentionArgs &a, bool whole, int workers, hipStream_t stream)
{
    switch (a.dim) {
    case 64: return attention_of<Type, E4M3, 64>(a, whole, workers, stream);
    case 96: return attention_of<Type, E4M3, 96>(a, whole, workers, stream);
    case 128: return attention_of<Type, E4M3, 128>(a, whole, workers, stream);
    case 192: return attention_of<Type, E4M3, 192>(a, whole, workers, stream);
    default: return attention_of<Type, E4M3, 256>(a, whole, workers, stream);
    }
}

}  // namespace

int64_t attention_units(int32_t max_pages, int32_t page_size)
{
    return ((int64_t)max_pages * page_size + kUnit - 1) / kUnit + 1;   // a window may start inside one
}

int64_t attention_workspace(int32_t, int32_t, int32_t dim)
{
    return (int64_t)2 * kMaxWorkers * 16 * (dim + 2) * sizeof(float) + kMaxWorkers * sizeof(Ending);
}

hipError_t launch_attention(const AttentionArgs &a, int cus, hipStream_t stream)
{
    // Two work-groups per CU are resident; never more than there can be units.
    const int share = a.Hq / a.Hkv;
    const int64_t groups = (int64_t)a.Hkv * ((share + 15) / 16);
    const int64_t units = attention_units(a.max_pages, a.page_size);
    int64_t workers = 2 * cus < kMaxWorkers ? 2 * cus : kMaxWorkers;
    if (units * groups * a.B < workers)
        workers = units * groups * a.B;
    // Row addresses inside a half tile are 32-bit offsets from a uniform base.
    const int64_t most = (1LL << 31) / 64;
    const bool whole = a.page_size % 16 == 0 && a.k_slot >= 0 && a.k_slot < most && a.v_slot >= 0 && a.v_slot < most;
    if (a.e4m3)
        a.type ? attention_dim<Fp16, true>(a, whole, (int)workers, stream)
               : attention_dim<Bf16, true>(a, whole, (int)workers, stream);
    else
        a.type ? attention_dim<Fp16, false>(a, whole, (int)workers, stream)
               : attention_dim<Bf16, false>(a, whole, (int)workers, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (units <= 2 && !a.window)   // one unit per head at most: nothing is split
        return hipSuccess;
    a.type ? join_kernel<Fp16><<<dim3((unsigned)workers), dim3(kJoinThreads), 0, stream>>>(a)
           : join_kernel<Bf16><<<dim3((unsigned)workers), dim3(kJoinThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a16
