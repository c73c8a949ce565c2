// Attention of one new token per request over a paged cache of 8-bit codes with a scale for each block of
// tokens and head, for gfx950: with keys ks_b c and values vs_b d (c, d codes, b a position's block),
//   s_j = scale * ks_b q . c_j,   out = sum_j e^{s_j} vs_b d_j / sum_j e^{s_j}.
//
// Work, split and operands are those of attention over 16-bit caches: equal runs of units of 128 positions, a
// wave taking every fourth tile of 32, S^T = K Q^T and O^T = V^T P^T, pieces joined by a second launch. Blocks
// are multiples of 16 positions, so each half of a tile has one scale for keys and one for values, which the
// lanes look up with the pages, for 32 tiles at a time.
//
// Products run in float16, which holds every code exactly, and so do bfloat16 queries, times a power of two that
// brings the head's largest magnitude to 2^15 (8 bits down to 2^-32 of it). An int8 code becomes float16 by a byte
// permute, which makes 1024 + 128 + code of it, and one packed subtraction: 5 operations for 4 codes.
//
// A value's scale goes with its weight, e^{s_j} vs_b, and float16 has little range: the reference of these
// weights is the running maximum of s_j + log vs_b, less 15 powers of two. They enter as two float16 values (22 bits
// down to 2^-18 of the largest one): with one, float16 outputs were off by 2.74e-4 of their norm where their own
// rounding is 2.06e-4 (48 requests of up to 5000), for 85.4 us instead of 87.1 (64 ragged requests of up to 8192). The
// weights' own sum has another reference, the maximum of s_j, and is held in float32 without rounding.
//
// The cache's bytes bound it. 64 ragged requests of up to 8192 positions, 64 heads on 8 of 128, int8: 83 us and 5 joining
// (medians of a trace; 87 in all by events; 0.44 GB: 5.3 TB/s here, where a streaming read of 4 GiB reaches 6.3); one
// request of 131000 positions 55 and 8 us, of 1100 7.0 and 4; 48 requests of up to 5000, e4m3, 26 and 5. By events, with
// one value of the weights, three work-groups per CU 87.9 us instead of 84.9, four 133; V a tile ahead as well as K 86
// instead of 85.
#include "attention_runs.h"

namespace w4a16 {

namespace {

// ---- one tile's operands -------------------------------------------------------------------------

constexpr float kHeadroom = 15.0f;

// Two codes (bytes 0 and 1, or 2 and 3) as float16 values, exactly. int8 codes come with their sign bit flipped.
template <bool INT8, bool HI>
__device__ __forceinline__ uint32_t from_codes(uint32_t w)
{
    if constexpr (INT8) {
        const uint32_t x = __builtin_amdgcn_perm(0x64646464u, w, HI ? 0x04030402u : 0x04010400u);
        const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) - bias);
    } else {
        return from_e4m3<HI>(Fp16(), w);
    }
}
template <bool INT8>
__device__ __forceinline__ uint32_t flipped(uint32_t w) { return INT8 ? w ^ 0x80808080u : w; }

template <bool INT8, int D>
struct CodeKeys {   // one half tile: 16 positions
    uint32_t w[D / 32][2];
    __device__ __forceinline__ void load(const uint8_t *p, int g)
    {
        typedef KeyDims<D, true> KD;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            if (c >= KD::paired) {
                const u32x2 x = __builtin_nontemporal_load((const u32x2 *)(p + KD::dim(c, g)));
                w[c][0] = x[0]; w[c][1] = x[1];
            } else if (c % 2 == 0) {
                const u32x4 x = __builtin_nontemporal_load((const u32x4 *)(p + KD::dim(c, g)));
                w[c][0] = x[0]; w[c][1] = x[1]; w[c + 1][0] = x[2]; w[c + 1][1] = x[3];
            }
        }
    }
    __device__ __forceinline__ u32x4 operand(int c) const
    {
        const uint32_t x = flipped<INT8>(w[c][0]), y = flipped<INT8>(w[c][1]);
        return u32x4{from_codes<INT8, false>(x), from_codes<INT8, true>(x), from_codes<INT8, false>(y),
                     from_codes<INT8, true>(y)};
    }
};

// The codes of one V row, as Parts has them: word x holds those of local values 4x .. (two in the last for 96).
template <int D>
struct CodeRow {
    static constexpr int head = Parts<D>::first / 4, words = (D / 16 + 3) / 4;
    uint32_t w[words];
    __device__ __forceinline__ void load(const uint8_t *p, const uint8_t *q)
    {
        load_part<Parts<D>::first, true>(p, w);
        if constexpr (Parts<D>::second > 0)
            load_part<Parts<D>::second, true>(q, w + head);
    }
};

// Where a wave's tiles lie and their scales: a lane holds those of one half tile, for 32 tiles of the wave at a
// time. Positions that are not read (outside lo..n-1, or on a page that is none) have offset 0, which is in the
// cache, and their bit of `live` is 0.
struct Halves {
    int64_t k, v;             // this lane's half tile: byte offsets
    float ks, vs;             // and scales
    uint64_t fine;            // lanes whose page is one of the cache
    uint32_t live;            // bit i: position i of the tile is read
    int64_t k0, k1, v0, v1;   // the tile's
    float ks0, ks1, vs0, vs1;

    // Tile number `i` of the wave, at position j0 = start + i * kUnit.
    __device__ __forceinline__ void go(const QuantizedAttentionArgs &a, const Head &h, const Span &s, int start, int i)
    {
        const int lane = threadIdx.x & 63;
        const int64_t j0 = (int64_t)start + (int64_t)i * kUnit;
        const int64_t below = s.lo - j0, above = s.n - j0;   // positions of the tile: below <= . < above
        uint32_t in = above >= 32 ? ~0u : above <= 0 ? 0u : (1u << above) - 1;
        in &= below <= 0 ? ~0u : below >= 32 ? 0u : ~0u << below;
        if ((i & 31) == 0) {
            const int64_t j = j0 + (int64_t)(lane >> 1) * kUnit + (lane & 1) * 16;
            const uint32_t at = (uint32_t)j / (uint32_t)a.page_size, slot = (uint32_t)j - at * (uint32_t)a.page_size;
            int32_t page = -1;
            if (j < s.n && j + 16 > s.lo)
                page = a.table[h.b * a.row_stride + at];
            const bool ok = page >= 0 && page < a.num_pages;
            k = v = 0;
            ks = vs = 1.0f;
            if (ok) {
                const uint32_t block = slot / (uint32_t)a.block;
                k = page * a.k_page + slot * a.k_slot;
                v = page * a.v_page + slot * a.v_slot;
                ks = a.k_scale[page * a.k_scale_page + block * a.k_scale_block + h.kv * a.k_scale_head];
                vs = a.v_scale[page * a.v_scale_page + block * a.v_scale_block + h.kv * a.v_scale_head];
            }
            fine = __ballot(ok);
        }
        const int at = 2 * (i & 31);
        auto read32 = [](float x, int l) {
            return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
        };
        k0 = read64(k, at);
        k1 = read64(k, at + 1);
        v0 = read64(v, at);
        v1 = read64(v, at + 1);
        ks0 = read32(ks, at);
        ks1 = read32(ks, at + 1);
        vs0 = read32(vs, at);
        vs1 = read32(vs, at + 1);
        const uint32_t two = (uint32_t)(fine >> at);
        live = in & ((two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u));
    }
};

// A head's queries as float16, and the power of two that they were divided by.
template <int D>
struct Queries {
    u32x4 w[D / 32];
    float back;
    __device__ __forceinline__ void load(const QuantizedAttentionArgs &a, const Head &head, int64_t b, int col, int g)
    {
        back = 1.0f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            w[c] = u32x4{0, 0, 0, 0};
            if (col < head.heads)
                w[c] = *(const u32x4 *)((const uint16_t *)a.q + b * a.ldq + (head.h0 + col) * a.hsq +
                                        KeyDims<D, true>::dim(c, g));
        }
        if (a.type)   // float16 as it is
            return;
        float most = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                most = fmaxf(most, fmaxf(fabsf(__builtin_bit_cast(float, w[c][e] << 16)),
                                         fabsf(__builtin_bit_cast(float, w[c][e] & 0xFFFF0000u))));
        most = max4(most);
        const int up = most > 0.0f && most < INFINITY ? min(15 - __builtin_amdgcn_frexp_expf(most), 120) : 0;
        back = __builtin_ldexpf(1.0f, -up);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[c][e] = pack2(Fp16(), __builtin_ldexpf(__builtin_bit_cast(float, w[c][e] << 16), up),
                                __builtin_ldexpf(__builtin_bit_cast(float, w[c][e] & 0xFFFF0000u), up));
    }
};

__device__ __forceinline__ float max8(const float *x)
{
    float m = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e)
        m = fmaxf(m, x[e]);
    return m;
}

template <bool INT8, int D>
__global__ __launch_bounds__(kThreads, 2) void quantized_attention_kernel(QuantizedAttentionArgs a)
{
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
    const uint32_t k_lane = (uint32_t)(col * a.k_slot), v_lane = (uint32_t)(4 * g * a.v_slot);
    const uint32_t first = P::first * col, second = 16 * P::first + P::second * col;
    const float to_log2 = a.scale * kLog2e;

    while (u < place.u1) {
        const uint32_t count = min(place.u1 - u, span.units - t0);
        const Head head = head_of(a, b, group);
        const uint8_t *kb = (const uint8_t *)a.k + head.kv * a.k_head;
        const uint8_t *vb = (const uint8_t *)a.v + head.kv * a.v_head;
        const int start = span.base + (int)(t0 * kUnit) + wave * kTile;
        // tiles of this wave: the last unit may end before this wave's tile of it
        int tiles = (int)count;
        if (tiles && (int64_t)start + (int64_t)(tiles - 1) * kUnit >= span.n)
            --tiles;

        Queries<D> q;
        CodeKeys<INT8, D> keys[2];
        CodeRow<D> rows[8];
        Halves r;
        auto load_keys = [&]() {
            keys[0].load(kb + r.k0 + k_lane, g);
            keys[1].load(kb + r.k1 + k_lane, g);
        };
        f32x4 o[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float top = -INFINITY, total = 0.0f;   // total: this lane's positions only, until the end
        float o_top = -INFINITY;               // reference of o
        if (tiles) {
            r.go(a, head, span, start, 0);
            load_keys();
        }
        q.load(a, head, b, col, g);
        for (int i = 0; i < tiles; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint8_t *p = vb + (e < 4 ? r.v0 : r.v1) + (e & 3) * a.v_slot + v_lane;
                rows[e].load(p + first, p + second);
            }
            const uint32_t live = r.live;
            const float ks[2] = {r.ks0 * q.back, r.ks1 * q.back}, vs[2] = {r.vs0, r.vs1};
            __builtin_amdgcn_sched_barrier(0);
            f32x4 s[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                s[half] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    s[half] = mfma(Fp16(), keys[half].operand(c), q.w[c], s[half]);
            }
            if (i + 1 < tiles) {
                r.go(a, head, span, start, i + 1);
                load_keys();
            }
            __builtin_amdgcn_sched_barrier(0);
            float x[8], y[8];   // scores, and with the values' scales: powers of two
            const float lift[2] = {__builtin_amdgcn_logf(vs[0]), __builtin_amdgcn_logf(vs[1])};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = s[e >> 2][e & 3] * ks[e >> 2] * to_log2;
                y[e] = x[e] + lift[e >> 2];
            }
            if (live != ~0u) {   // positions that are not read: no weight, and no value either
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!((live >> ((e < 4 ? 0 : 12) + 4 * g + e)) & 1)) {
                        x[e] = y[e] = -INFINITY;
#pragma unroll
                        for (int w = 0; w < CodeRow<D>::words; ++w)
                            rows[e].w[w] = 0;
                    }
            }
            const float m = fmaxf(max4(max8(x)), top), ref = m == -INFINITY ? 0.0f : m;   // nothing seen yet: weights 0
            const float o_m = fmaxf(max4(max8(y)) - kHeadroom, o_top), o_ref = o_m == -INFINITY ? 0.0f : o_m;
            const float fade = __builtin_amdgcn_exp2f(o_top - o_ref);
            total *= __builtin_amdgcn_exp2f(top - ref);
            top = m;
            o_top = o_m;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                total += __builtin_amdgcn_exp2f(x[e] - ref);
                y[e] = __builtin_amdgcn_exp2f(y[e] - o_ref);
            }
            u32x4 p, rest;   // the weights with the values' scales, at most 2^15, as float16, and what that leaves
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t both = pack2(Fp16(), y[2 * e], y[2 * e + 1]);
                asm volatile("" : "+v"(both));   // or the remainder converts once more
                const f16x2 x = __builtin_bit_cast(f16x2, both);
                p[e] = both;
                rest[e] = pack2(Fp16(), y[2 * e] - (float)x[0], y[2 * e + 1] - (float)x[1]);
            }
            if (__ballot(fade != 1.0f)) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[j][k] *= fade;
            }
#pragma unroll
            for (int w = 0; w < CodeRow<D>::words; ++w) {
                u32x4 v[4];   // values 4w .. of the eight rows, rows in pairs
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t r0 = rows[2 * e].w[w], r1 = rows[2 * e + 1].w[w];
                    const uint32_t lo = flipped<INT8>(__builtin_amdgcn_perm(r1, r0, 0x05010400u));
                    const uint32_t hi = flipped<INT8>(__builtin_amdgcn_perm(r1, r0, 0x07030602u));
                    v[0][e] = from_codes<INT8, false>(lo);
                    v[1][e] = from_codes<INT8, true>(lo);
                    v[2][e] = from_codes<INT8, false>(hi);
                    v[3][e] = from_codes<INT8, true>(hi);
                }
#pragma unroll
                for (int j = 4 * w; j < 4 * w + 4 && j < D / 16; ++j)
                    o[j] = mfma(Fp16(), v[j & 3], p, o[j]);
                __builtin_amdgcn_sched_barrier(0);   // 47 scalars spilled instead of 78: one request of 1100 11.0 -> 10.6 us
#pragma unroll
                for (int j = 4 * w; j < 4 * w + 4 && j < D / 16; ++j)
                    o[j] = mfma(Fp16(), v[j & 3], rest, o[j]);
            }
        }

        // Join the four waves in LDS. A lane holds, of head col, dims of V lane 4g + k (k < 4).
        total = sum4(total);
        // One reference again, in two halves: exp2 gives zero below 2^-126, and value scales go down to that themselves.
        const float half_even = o_top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(0.5f * (o_top - top));
        __syncthreads();   // the scan's sums, or the previous piece's, have been read
        if (g == 0) {
            tops[wave][col] = top;
            totals[wave][col] = total;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < D / 16; j += 2)
                *(f32x2 *)&sums[wave][col][P::dim(4 * g + k, j)] =
                    f32x2{o[j][k] * half_even * half_even, o[j + 1][k] * half_even * half_even};
        __syncthreads();
        const bool whole = t0 == 0 && count == span.units;
        const int piece = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
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
                const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = l == 0.0f ? 0.0f : sum[e] * f;
                a.type ? store_out<Fp16>(a, b, head.h0 + h, d, sum) : store_out<Bf16>(a, b, head.h0 + h, d, sum);
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

template <bool INT8>
void quantized_dim(const QuantizedAttentionArgs &a, int workers, hipStream_t stream)
{
    const dim3 grid((unsigned)workers), block(kThreads);
    switch (a.dim) {
    case 64: quantized_attention_kernel<INT8, 64><<<grid, block, 0, stream>>>(a); break;
    case 96: quantized_attention_kernel<INT8, 96><<<grid, block, 0, stream>>>(a); break;
    case 128: quantized_attention_kernel<INT8, 128><<<grid, block, 0, stream>>>(a); break;
    case 192: quantized_attention_kernel<INT8, 192><<<grid, block, 0, stream>>>(a); break;
    default: quantized_attention_kernel<INT8, 256><<<grid, block, 0, stream>>>(a); break;
    }
}

}  // namespace

hipError_t launch_quantized_attention(const QuantizedAttentionArgs &a, int cus, hipStream_t stream)
{
    // Two work-groups per CU are resident; never more than there can be units.
    const int share = a.Hq / a.Hkv;
    const int64_t groups = (int64_t)a.Hkv * ((share + 15) / 16);
    const int64_t units = attention_units(a.max_pages, a.page_size);
    int64_t workers = 2 * cus < kMaxWorkers ? 2 * cus : kMaxWorkers;
    if (units * groups * a.B < workers)
        workers = units * groups * a.B;
    a.int8 ? quantized_dim<true>(a, (int)workers, stream) : quantized_dim<false>(a, (int)workers, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (units <= 2 && !a.window))   // one unit per head at most: nothing is split
        return e;
    const AttentionArgs &join = a;
    a.type ? join_kernel<Fp16><<<dim3((unsigned)workers), dim3(kJoinThreads), 0, stream>>>(join)
           : join_kernel<Bf16><<<dim3((unsigned)workers), dim3(kJoinThreads), 0, stream>>>(join);
    return hipGetLastError();
}

}  // namespace w4a16
